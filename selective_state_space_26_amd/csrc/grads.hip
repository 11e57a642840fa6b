// grads.hip -- the norm over all gradients of a model and the gradients scaled to a bound on it:
//   norm = sqrt(sum g^2),  out = g min(1, max_norm / (norm + eps)).
//
// HBM bounds it: the tensors are read for the norm and, after it is known, read and written for
// the scaling.  Every launch takes up to kTable tensors in its arguments (no table in device
// memory, nothing kept between calls), each cut into chunks of the same length; a block sums one
// chunk in fp64 (a square of an fp32 value neither overflows nor vanishes there, and the chip's
// fp64 rate is far above what HBM delivers) into one partial sum.  The partial sums are
// added in a fixed order: deterministic.  The scaling walks the chunks from the last to the
// first: what the norm read last is still in the last-level cache, and outputs larger than it go
// past it (129 M fp32 values: 273 us, 301 through the cache).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lm_device.hpp"
#include "lm_kernels.hpp"

namespace msel {

namespace {

constexpr int kTable = 128;
constexpr int64_t kMinChunk = 8192;  // elements: 4 rounds of a block's vectors in bf16, 8 in fp32
// Chunks over all tensors: many rounds of blocks, so that CUs end together (129 M fp32 values:
// 345 us with 2048, 302 with 16384).
constexpr int64_t kTargetChunks = 16384;
// Up to this many partial sums every scaling block adds them itself (a few loads per thread),
// which saves the launch in between: 90 tensors of 0.26 M values 19.6 us with it, 16 without.
constexpr int64_t kSelfSum = 1024;

struct GradTable {
    const void* src[kTable];
    void* dst[kTable];
    int64_t n[kTable];              // elements, bf16 tensors as -n
    uint32_t start[kTable];         // first chunk of the entry in this launch
    int count;
    uint32_t chunks;                // in this launch
    int64_t chunk;                  // elements
    int64_t base;                   // first chunk of this launch among all
};
static_assert(sizeof(GradTable) + 64 <= 4096, "a kernel's arguments");

// The entry whose chunks hold chunk c: the last with start <= c.
__device__ __forceinline__ int entry_of(const GradTable& t, uint32_t c) {
    int k = 0;
#pragma unroll
    for (int j = 0; j < kTable; j += 64) {
        const int l = j + lane_id();
        k += __popcll(__ballot(l < t.count && t.start[l] <= c));
    }
    return k - 1;
}

template <typename T>
__device__ __forceinline__ double chunk_sum(const T* p, int64_t n) {
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    constexpr int UN = 4;
    double s[2] = {0.0, 0.0};
    const int64_t nv = n / VE;
    const auto add = [&](const RawVec<T, VE>& r) {
        float v[VE];
        to_f32<T, VE>(r, v);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const double d = static_cast<double>(v[k]);
            s[k & 1] = fma(d, d, s[k & 1]);
        }
    };
    int64_t i = threadIdx.x;
    for (; i + 256 * (UN - 1) < nv; i += 256 * UN) {
        RawVec<T, VE> r[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) r[u] = ld_raw<T, VE>(p + MSEL_SPAN((i + 256 * u) * VE, VE, n));
#pragma unroll
        for (int u = 0; u < UN; ++u) add(r[u]);
    }
    for (; i < nv; i += 256) add(ld_raw<T, VE>(p + MSEL_SPAN(i * VE, VE, n)));
    if (threadIdx.x < n - nv * VE) {
        const double d = static_cast<double>(Elem<T>::load1(p + MSEL_IDX(nv * VE + threadIdx.x, n)));
        s[0] = fma(d, d, s[0]);
    }
    return s[0] + s[1];
}

// Sum over a block, in thread 0; red: one double per wavefront.
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int m = 32; m > 0; m /= 2) v += __shfl_xor(v, m);
    if (lane_id() == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < WAVES; ++w) v += red[w];
    return v;
}

__global__ __launch_bounds__(256) void grad_sums_kernel(GradTable t, double* partials,
                                                        int64_t total) {
    __shared__ double red[4];
    const uint32_t c = blockIdx.x;
    const int e = __builtin_amdgcn_readfirstlane(entry_of(t, c));
    const int64_t len = t.n[e] < 0 ? -t.n[e] : t.n[e];
    const int64_t i0 = static_cast<int64_t>(c - t.start[e]) * t.chunk;
    const int64_t n = min(t.chunk, len - i0);
    const double s = t.n[e] < 0 ? chunk_sum(static_cast<const bf16_t*>(t.src[e]) + i0, n)
                                : chunk_sum(static_cast<const float*>(t.src[e]) + i0, n);
    const double v = block_sum<4>(s, red);
    if (threadIdx.x == 0) partials[MSEL_IDX(t.base + c, total)] = v;
}

// min(1, max_norm / (norm + eps)); a NaN stays.
__device__ __forceinline__ float factor_of(float norm, float max_norm, float eps) {
    const float q = max_norm / (norm + eps);
    return q >= 1.0f ? 1.0f : q;
}

// norm and, behind the partial sums, the scaling factor.
__global__ __launch_bounds__(1024) void grad_norm_kernel(double* partials, int64_t total,
                                                         float max_norm, float eps, float* norm) {
    __shared__ double red[16];
    double s = 0.0;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < total; i += 1024) s += partials[i];
    s = block_sum<16>(s, red);
    if (threadIdx.x == 0) {
        const float nrm = static_cast<float>(sqrt(s));
        *norm = nrm;
        reinterpret_cast<float*>(partials + total)[0] = factor_of(nrm, max_norm, eps);
    }
}

template <bool PAST, typename T>
__device__ __forceinline__ void chunk_scale(const T* p, T* q, int64_t n, float f) {
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    constexpr int UN = 4;
    const int64_t nv = n / VE;
    const auto put = [&](int64_t i, const RawVec<T, VE>& r) {
        float v[VE];
        to_f32<T, VE>(r, v);
#pragma unroll
        for (int k = 0; k < VE; ++k) v[k] *= f;
        st_vec<T, VE, PAST>(q + MSEL_SPAN(i * VE, VE, n), v);
    };
    int64_t i = threadIdx.x;
    for (; i + 256 * (UN - 1) < nv; i += 256 * UN) {
        RawVec<T, VE> r[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) r[u] = ld_raw<T, VE>(p + MSEL_SPAN((i + 256 * u) * VE, VE, n));
#pragma unroll
        for (int u = 0; u < UN; ++u) put(i + 256 * u, r[u]);
    }
    for (; i < nv; i += 256) put(i, ld_raw<T, VE>(p + MSEL_SPAN(i * VE, VE, n)));
    if (threadIdx.x < n - nv * VE) {
        const int64_t j = MSEL_IDX(nv * VE + threadIdx.x, n);
        Elem<T>::store1(q + j, Elem<T>::load1(p + j) * f);
    }
}

// PAST: outputs go past the caches, so that they push out no gradient that is still to be read.
// total > 0: the factor is made here from that many partial sums, and block 0 of the launch that
// has `norm` writes it.
template <bool PAST>
__global__ __launch_bounds__(256) void grad_scale_kernel(GradTable t, const double* partials,
                                                         int64_t total, const float* factor,
                                                         float max_norm, float eps, float* norm) {
    __shared__ double red[4];
    __shared__ float shared_f;
    const uint32_t c = t.chunks - 1 - blockIdx.x;
    float f;
    if (total > 0) {  // grid-uniform
        double s = 0.0;
#pragma unroll 4
        for (int64_t i = threadIdx.x; i < total; i += 256) s += partials[i];
        s = block_sum<4>(s, red);
        if (threadIdx.x == 0) {
            const float nrm = static_cast<float>(sqrt(s));
            if (norm != nullptr && blockIdx.x == 0) *norm = nrm;
            shared_f = factor_of(nrm, max_norm, eps);
        }
        __syncthreads();
        f = shared_f;
    } else {
        f = *factor;
    }
    const int e = __builtin_amdgcn_readfirstlane(entry_of(t, c));
    if (f == 1.0f && t.src[e] == t.dst[e]) return;  // in place, and every value stays
    const int64_t len = t.n[e] < 0 ? -t.n[e] : t.n[e];
    const int64_t i0 = static_cast<int64_t>(c - t.start[e]) * t.chunk;
    const int64_t n = min(t.chunk, len - i0);
    if (t.n[e] < 0)
        chunk_scale<PAST>(static_cast<const bf16_t*>(t.src[e]) + i0,
                          static_cast<bf16_t*>(t.dst[e]) + i0, n, f);
    else
        chunk_scale<PAST>(static_cast<const float*>(t.src[e]) + i0,
                          static_cast<float*>(t.dst[e]) + i0, n, f);
}

int64_t chunk_of(const GradNormParams& p) {
    int64_t total = 0;
    for (int i = 0; i < p.count; ++i) total += p.read(p.list, p.outs, i).n;
    const int64_t per = (total + kTargetChunks - 1) / kTargetChunks;
    return std::max<int64_t>(kMinChunk, (per + kMinChunk - 1) / kMinChunk * kMinChunk);
}

int64_t out_bytes(const GradNormParams& p) {
    int64_t bytes = 0;
    for (int i = 0; i < p.count; ++i) {
        const GradTensor g = p.read(p.list, p.outs, i);
        bytes += g.n * (g.bf16 ? 2 : 4);
    }
    return bytes;
}

}  // namespace

int64_t grad_partials(const GradNormParams& p) {
    const int64_t chunk = chunk_of(p);
    int64_t n = 0;
    for (int i = 0; i < p.count; ++i) n += (p.read(p.list, p.outs, i).n + chunk - 1) / chunk;
    return n;
}

hipError_t launch_grad_norm(const GradNormParams& p, bool clip, hipStream_t stream) {
    const int64_t chunk = chunk_of(p), total = grad_partials(p);
    const float* factor = reinterpret_cast<const float*>(p.partials + total);
    const bool self = clip && total > 0 && total <= kSelfSum;
    float* norm = self ? p.norm : nullptr;
    const bool past = past_cache(out_bytes(p));
    for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
        int i = pass == 0 ? 0 : p.count - 1;
        const int step = pass == 0 ? 1 : -1;
        int64_t base = 0;
        while (i >= 0 && i < p.count) {
            GradTable t;
            t.count = 0;
            t.chunks = 0;
            t.chunk = chunk;
            t.base = base;
            // the scaling takes the tensors, and below a launch's chunks, from the last on
            for (; i >= 0 && i < p.count && t.count < kTable; i += step) {
                const GradTensor g = p.read(p.list, p.outs, i);
                if (g.n == 0) continue;
                t.src[t.count] = g.src;
                t.dst[t.count] = g.dst;
                t.n[t.count] = g.bf16 ? -g.n : g.n;
                t.start[t.count++] = t.chunks;
                t.chunks += static_cast<uint32_t>((g.n + chunk - 1) / chunk);
            }
            if (t.count == 0) break;
            if (pass == 0)
                hipLaunchKernelGGL(grad_sums_kernel, dim3(t.chunks), dim3(256), 0, stream, t,
                                   p.partials, total);
            else
                hipLaunchKernelGGL(past ? grad_scale_kernel<true> : grad_scale_kernel<false>,
                                   dim3(t.chunks), dim3(256), 0, stream, t, p.partials,
                                   self ? total : 0, factor, p.max_norm, p.eps, norm);
            if (pass == 1) norm = nullptr;  // the first launch writes it
            base += t.chunks;
        }
        if (pass == 0 && !self)
            hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(1024), 0, stream, p.partials, total,
                               p.max_norm, p.eps, p.norm);
    }
    return hipGetLastError();
}

MSEL_BOUNDS_TAKER(take_bounds_grads)

}  // namespace msel
