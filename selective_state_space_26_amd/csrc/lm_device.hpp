// lm_device.hpp -- device-side building blocks of the operators around the scan (norms,
// embedding, gradient clipping).
//
// Rows of these operators need not be multiples of a vector: a row of an odd width starts at
// any element.  ld_vec / st_vec move 16 or 8 bytes at element alignment as one instruction
// (global accesses on gfx950 need no more than element alignment), so that only the last
// width % VE elements of a row take element-wise accesses.
#pragma once

#include "msel_device.hpp"

namespace msel {

// A span of w elements starting at i inside an extent of n: the checked build counts a span
// that leaves [0, n) and moves it to 0 (spans are only formed where n >= w).
#ifdef MSEL_CHECKED
template <typename I>
__device__ __forceinline__ I checked_span(I i, long long w, unsigned long long n,
                                          unsigned int line) {
    const long long s = static_cast<long long>(i);
    if (s >= 0 && static_cast<unsigned long long>(s + w) <= n) return i;
    checked_index(-1, n, line);
    return I(0);
}
#define MSEL_SPAN(i, w, n) \
    ::msel::checked_span((i), (w), static_cast<unsigned long long>(n), __LINE__)
#else
#define MSEL_SPAN(i, w, n) (i)
#endif

template <int BYTES> struct Words;
template <> struct Words<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <> struct Words<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };
template <> struct Words<32> { typedef uint32_t type __attribute__((ext_vector_type(8))); };

// VE elements as they lie in memory.
template <typename T, int VE>
struct RawVec {
    typename Words<VE * static_cast<int>(sizeof(T))>::type w;
};

template <typename T, int VE>
__device__ __forceinline__ RawVec<T, VE> ld_raw(const T* p) {
    RawVec<T, VE> r;
    __builtin_memcpy(&r.w, p, sizeof(r.w));
    return r;
}

template <typename T, int VE>
__device__ __forceinline__ void to_f32(const RawVec<T, VE>& r, float (&v)[VE]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < VE; ++k) v[k] = __uint_as_float(r.w[k]);
    } else {
#pragma unroll
        for (int k = 0; k < VE; k += 2) {
            v[k] = bf16lo(r.w[k / 2]);
            v[k + 1] = bf16hi(r.w[k / 2]);
        }
    }
}

template <typename T, int VE>
__device__ __forceinline__ RawVec<T, VE> from_f32(const float (&v)[VE]) {
    RawVec<T, VE> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < VE; ++k) r.w[k] = __float_as_uint(v[k]);
    } else {
#pragma unroll
        for (int k = 0; k < VE; k += 2) r.w[k / 2] = pack_bf16(v[k], v[k + 1]);
    }
    return r;
}

// PAST: a store past the caches, for outputs that leave them before anyone reads them anyway
// (past_cache below).
template <typename T, int VE, bool PAST = false>
__device__ __forceinline__ void st_raw(T* p, const RawVec<T, VE>& r) {
    if constexpr (PAST) {
        typedef typename Words<VE * static_cast<int>(sizeof(T))>::type U
            __attribute__((aligned(sizeof(T))));
        __builtin_nontemporal_store(r.w, reinterpret_cast<U*>(p));
    } else {
        __builtin_memcpy(p, &r.w, sizeof(r.w));
    }
}

template <typename T, int VE, bool PAST = false>
__device__ __forceinline__ void st_vec(T* p, const float (&v)[VE]) {
    st_raw<T, VE, PAST>(p, from_f32<T, VE>(v));
}

// The first `valid` of VE elements at p (the rest 0): element by element unless all are valid.
template <typename T, int VE>
__device__ __forceinline__ RawVec<T, VE> ld_part(const T* p, int valid) {
    if (valid >= VE) return ld_raw<T, VE>(p);
    float v[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) v[k] = k < valid ? Elem<T>::load1(p + k) : 0.0f;
    return from_f32<T, VE>(v);
}

template <typename T, int VE, bool PAST = false>
__device__ __forceinline__ void st_part(T* p, const RawVec<T, VE>& r, int valid) {
    if (valid >= VE) {
        st_raw<T, VE, PAST>(p, r);
        return;
    }
    float v[VE];
    to_f32<T, VE>(r, v);
#pragma unroll
    for (int k = 0; k < VE; ++k)
        if (k < valid) Elem<T>::store1(p + k, v[k]);
}

// Whether an output of so many bytes is stored past the caches: beyond half of the last-level
// cache (256 MiB) little of it would be there for its reader, and what it pushes out is read again
// (inputs whose lines are shared by tiles, gradients between norm and scaling).
inline bool past_cache(int64_t bytes) { return bytes > (int64_t(128) << 20); }

// Consecutive tiles on one XCD: blocks go to the 8 XCDs in turn, and neighbouring tiles share
// cache lines wherever a tile's rows do not start and end on one.
__device__ __forceinline__ unsigned xcd_order(unsigned bid, unsigned n) {
    const unsigned x = bid & 7u, q = n >> 3, r = n & 7u;
    return x * q + (x < r ? x : r) + (bid >> 3);
}

// Tiles over a grid: a grid's dimension has fewer than 2^32 threads, so that tiles beyond kGridX
// go on along z (the last slice may have blocks without a tile).
constexpr unsigned kGridX = 1u << 21;
inline dim3 tile_grid(unsigned tiles, unsigned groups) {
    return tiles <= kGridX ? dim3(tiles, groups) : dim3(kGridX, groups, (tiles + kGridX - 1) / kGridX);
}
__device__ __forceinline__ int tile_of_block() {
    return static_cast<int>(blockIdx.z * gridDim.x + xcd_order(blockIdx.x, gridDim.x));
}

// silu(z) = z sigmoid(z) and its derivative sigmoid(z) (1 + z (1 - sigmoid(z))).
__device__ __forceinline__ float silu_f(float z) { return z * sigmoid_f(z); }
__device__ __forceinline__ void silu_grad_f(float z, float& gate, float& slope) {
    const float s = sigmoid_f(z);
    gate = z * s;
    slope = fmaf(gate, 1.0f - s, s);
}

// 1 / sqrt(mean square + eps) from the sum of n squares.
__device__ __forceinline__ float rstd_of(float sum_sq, float inv_n, float eps) {
    return 1.0f / sqrtf(fmaf(sum_sq, inv_n, eps));
}

}  // namespace msel
