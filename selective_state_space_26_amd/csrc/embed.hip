// embed.hip -- embedding lookup with a scale, and the table's gradient by sorted tokens.
//
// Forward: out[t] = scale w[ids[t]], a gather of rows: HBM bounds it (the distinct rows once,
// the output once).
//
// Backward: dw[v] = base[v] + scale * (sum of dout[t] over the tokens with ids[t] = v).  The
// table is far larger than the batch for real vocabularies, so most of the bytes are dw itself.
// Three steps:
//  1. a stable radix sort of (id, position), ids outside [0, vocab) and the padding id last.
//     Digits of up to 9 bits; a block counts and places a run of consecutive tokens, ranks within
//     a wavefront by ballots, so that the order is the tokens' own: deterministic.  The sort
//     needs few blocks and waits on latency, so the same launches fill dw (with base or 0) on
//     the remaining CUs;
//  2. segment sums: the sorted positions in chunks of kSeg entries; a team of lanes adds its
//     chunk's rows in fp32.  An id's run inside a chunk is written to dw directly; a run that
//     crosses chunks leaves one partial sum per chunk;
//  3. the partial sums of each crossing run are added in chunk order.
// No floating-point atomics, and a frequent id costs no more than a rare one.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lm_device.hpp"
#include "lm_kernels.hpp"

namespace msel {

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr int kMaxSortBlocks = 128;
constexpr int kFillBlocks = 512;
constexpr int kSeg = 32;         // sorted entries per segment-sum chunk
constexpr int kSegBatch = 8;     // of them in flight at a time

struct EmbedPlan {
    int passes, dbits, nblocks;
    int chunk;       // tokens per sort block
    int nseg;        // segment chunks
    size_t key[2], pos[2], table, partial, bytes;  // offsets into the workspace
};

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

EmbedPlan embed_plan(int64_t tokens, int vocab, int dim) {
    EmbedPlan pl{};
    int bits = 1;
    while ((int64_t(1) << bits) <= vocab) ++bits;  // the sentinel is vocab itself
    pl.passes = (bits + kDigitBits - 1) / kDigitBits;
    pl.dbits = (bits + pl.passes - 1) / pl.passes;
    const int64_t tiles = (tokens + kSortThreads - 1) / kSortThreads;
    const int64_t blocks = std::min<int64_t>(kMaxSortBlocks, tiles);
    pl.chunk = static_cast<int>((tiles + blocks - 1) / blocks * kSortThreads);
    pl.nblocks = static_cast<int>((tokens + pl.chunk - 1) / pl.chunk);
    pl.nseg = static_cast<int>((tokens + kSeg - 1) / kSeg);
    size_t at = 0;
    const auto take = [&](size_t n) {
        const size_t o = at;
        at += align256(n);
        return o;
    };
    for (int i = 0; i < 2; ++i) {
        pl.key[i] = take(static_cast<size_t>(tokens) * 4);
        pl.pos[i] = take(static_cast<size_t>(tokens) * 4);
    }
    pl.table = take(static_cast<size_t>(pl.passes) * kBins * pl.nblocks * 4);
    pl.partial = take(static_cast<size_t>(pl.nseg) * 2 * dim * 4);
    pl.bytes = at;
    return pl;
}

template <typename T, typename TW, int VE>
__global__ __launch_bounds__(256) void embed_fwd_kernel(EmbedParams p, int nvec, FastDiv by_nvec,
                                                        int block_tokens) {
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * block_tokens;
    const int nt = static_cast<int>(min(static_cast<int64_t>(block_tokens), p.tokens - t0));
    const uint32_t total = static_cast<uint32_t>(nt) * static_cast<uint32_t>(nvec);
    const T* const out0 = static_cast<const T*>(p.out);
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < total; i += 256) {
        const uint32_t dt = (__umulhi(i, by_nvec.m) + i) >> by_nvec.l;
        const int e0 = static_cast<int>(i - dt * static_cast<uint32_t>(nvec)) * VE;
        const int left = p.dim - e0;
        const int64_t t = MSEL_IDX(t0 + dt, p.tokens);
        const int64_t id = p.ids64 ? static_cast<const int64_t*>(p.ids)[t]
                                   : static_cast<const int32_t*>(p.ids)[t];
        float v[VE] = {};
        if (id >= 0 && id < p.vocab)
            to_f32<TW, VE>(ld_part<TW, VE>(static_cast<const TW*>(p.w) + id * p.dim + e0, left), v);
#pragma unroll
        for (int k = 0; k < VE; ++k) v[k] *= p.scale;
        st_part<T, VE>(const_cast<T*>(out0) + t * p.dim + e0, from_f32<T, VE>(v), left);
    }
}

// Elements [share s of n) of the fill of dw by base or 0: blocks j of `blocks`.
__device__ void fill_share(const EmbedParams& p, int share, int shares, int j, int blocks) {
    if (p.base == p.dw) return;  // added to in place
    const int64_t total = static_cast<int64_t>(p.vocab) * p.dim;
    const int64_t nv = total / 4;
    const int64_t v0 = nv / shares * share, v1 = share == shares - 1 ? nv : v0 + nv / shares;
    f32x4* d = reinterpret_cast<f32x4*>(p.dw);
    const f32x4* s = reinterpret_cast<const f32x4*>(p.base);
    const int64_t step = static_cast<int64_t>(blocks) * kSortThreads;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t i = v0 + static_cast<int64_t>(j) * kSortThreads + threadIdx.x; i < v1; i += step)
        d[MSEL_IDX(i, nv)] = s != nullptr ? s[i] : zero;
    if (share == shares - 1 && j == 0 && threadIdx.x < total - nv * 4) {
        const int64_t i = MSEL_IDX(nv * 4 + threadIdx.x, total);
        p.dw[i] = p.base != nullptr ? p.base[i] : 0.0f;
    }
}

// The sort key of token t: its id, or vocab for one that gives no gradient.
__device__ __forceinline__ uint32_t key_of(const EmbedParams& p, int64_t t) {
    const int64_t id = p.ids64 ? static_cast<const int64_t*>(p.ids)[t]
                               : static_cast<const int32_t*>(p.ids)[t];
    return id >= 0 && id < p.vocab && id != p.padding_idx ? static_cast<uint32_t>(id)
                                                          : static_cast<uint32_t>(p.vocab);
}

// Pass 0's digit counts per block, table[digit][block], and zeros for the later passes' tables.
__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(EmbedParams p, EmbedPlan pl) {
    __shared__ uint32_t cnt[kBins];
    if (static_cast<int>(blockIdx.x) >= pl.nblocks) {
        fill_share(p, 0, pl.passes + 1, blockIdx.x - pl.nblocks, gridDim.x - pl.nblocks);
        return;
    }
    uint32_t* table = reinterpret_cast<uint32_t*>(static_cast<char*>(p.ws) + pl.table);
    const int words = kBins * pl.nblocks;
    for (int i = threadIdx.x; i < kBins; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * pl.chunk;
    const int64_t t1 = min(t0 + pl.chunk, p.tokens);
    const uint32_t mask = (1u << pl.dbits) - 1u;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kSortThreads)
        atomicAdd(&cnt[MSEL_IDX(key_of(p, t) & mask, kBins)], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < kBins; d += kSortThreads) {
        const int at = d * pl.nblocks + static_cast<int>(blockIdx.x);
        table[MSEL_IDX(at, words)] = cnt[d];
        for (int q = 1; q < pl.passes; ++q) table[q * words + MSEL_IDX(at, words)] = 0;
    }
}

// Places the tokens of pass `pass` in digit order (stable), and counts the next pass's digits
// by destination block.
__global__ __launch_bounds__(kSortThreads) void embed_place_kernel(EmbedParams p, EmbedPlan pl,
                                                                   int pass) {
    __shared__ uint32_t run[kBins];               // next free place of each digit
    __shared__ uint32_t cnt[kSortWaves][kBins];
    if (static_cast<int>(blockIdx.x) >= pl.nblocks) {
        fill_share(p, pass + 1, pl.passes + 1, blockIdx.x - pl.nblocks, gridDim.x - pl.nblocks);
        return;
    }
    char* ws = static_cast<char*>(p.ws);
    const int words = kBins * pl.nblocks;
    const uint32_t* table = reinterpret_cast<const uint32_t*>(ws + pl.table) + pass * words;
    uint32_t* next = reinterpret_cast<uint32_t*>(ws + pl.table) + (pass + 1) * words;
    const uint32_t* key_in = reinterpret_cast<const uint32_t*>(ws + pl.key[(pass + 1) & 1]);
    const uint32_t* pos_in = reinterpret_cast<const uint32_t*>(ws + pl.pos[(pass + 1) & 1]);
    uint32_t* key_out = reinterpret_cast<uint32_t*>(ws + pl.key[pass & 1]);
    uint32_t* pos_out = reinterpret_cast<uint32_t*>(ws + pl.pos[pass & 1]);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int shift = pass * pl.dbits;
    const uint32_t mask = (1u << pl.dbits) - 1u;

    // where this block's tokens of each digit go: all smaller digits, then this digit in the
    // blocks before
    uint32_t total = 0, before = 0;
    if (tid < kBins) {
        for (int j = 0; j < pl.nblocks; ++j) {
            const uint32_t c = table[MSEL_IDX(tid * pl.nblocks + j, words)];
            total += c;
            before += j < static_cast<int>(blockIdx.x) ? c : 0u;
        }
        run[tid] = total;
    }
    __syncthreads();
    for (int s = 1; s < kBins; s *= 2) {
        const uint32_t v = tid < kBins && tid >= s ? run[tid - s] : 0u;
        __syncthreads();
        if (tid < kBins) run[tid] += v;
        __syncthreads();
    }
    if (tid < kBins) run[tid] += before - total;

    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * pl.chunk;
    const int64_t t1 = min(t0 + pl.chunk, p.tokens);
    for (int64_t tb = t0; tb < t1; tb += kSortThreads) {  // block-uniform
        for (int i = tid; i < kSortWaves * kBins; i += kSortThreads) (&cnt[0][0])[i] = 0;
        __syncthreads();
        const int64_t t = tb + tid;
        const bool in = t < t1;
        uint32_t key = 0, pos = 0;
        if (in) {
            key = pass == 0 ? key_of(p, t) : key_in[MSEL_IDX(t, p.tokens)];
            pos = pass == 0 ? static_cast<uint32_t>(t) : pos_in[MSEL_IDX(t, p.tokens)];
        }
        const uint32_t digit = (key >> shift) & mask;
        uint64_t same = __ballot(in);
        for (int bit = 0; bit < pl.dbits; ++bit) {
            const uint64_t b = __ballot((digit >> bit) & 1u);
            same &= (digit >> bit) & 1u ? b : ~b;
        }
        const int rank = __popcll(same & ((uint64_t(1) << lane) - 1u));
        if (in && rank == 0) cnt[wave][digit] = static_cast<uint32_t>(__popcll(same));
        __syncthreads();
        if (tid < kBins) {
            uint32_t s = run[tid];
            for (int w = 0; w < kSortWaves; ++w) {
                const uint32_t c = cnt[w][tid];
                cnt[w][tid] = s;
                s += c;
            }
            run[tid] = s;
        }
        __syncthreads();
        if (in) {
            const int64_t to = MSEL_IDX(static_cast<int64_t>(cnt[wave][digit] + rank), p.tokens);
            key_out[to] = key;
            pos_out[to] = pos;
            if (pass + 1 < pl.passes) {
                const uint32_t d2 = (key >> (shift + pl.dbits)) & mask;
                const int at = static_cast<int>(d2) * pl.nblocks + static_cast<int>(to / pl.chunk);
                atomicAdd(&next[MSEL_IDX(at, words)], 1u);
            }
        }
        __syncthreads();
    }
}

__device__ __forceinline__ void write_row(const EmbedParams& p, uint32_t v, int e0, int left,
                                          const float* acc, int ve) {
    const int64_t at = static_cast<int64_t>(MSEL_IDX(v, p.vocab)) * p.dim + e0;
    for (int k = 0; k < ve; ++k)
        if (k < left) {
            const float b = p.base != nullptr ? p.base[at + k] : 0.0f;
            p.dw[at + k] = fmaf(p.scale, acc[k], b);
        }
}

// Segment sums: a team of S lanes (S columns vectors of VE) per chunk of kSeg sorted entries.
template <typename T, int VE>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedParams p, EmbedPlan pl, int S,
                                                        int nvec) {
    const char* ws = static_cast<const char*>(p.ws);
    const uint32_t* key = reinterpret_cast<const uint32_t*>(ws + pl.key[(pl.passes - 1) & 1]);
    const uint32_t* pos = reinterpret_cast<const uint32_t*>(ws + pl.pos[(pl.passes - 1) & 1]);
    float* part = reinterpret_cast<float*>(static_cast<char*>(p.ws) + pl.partial);
    const int team = threadIdx.x / S, lane = threadIdx.x % S;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * (256 / S) + team;
    const int cv = blockIdx.y * S + lane;
    if (c >= pl.nseg || cv >= nvec) return;
    const int e0 = cv * VE, left = p.dim - e0;
    const int64_t i0 = c * kSeg;
    const int64_t i1 = min(i0 + kSeg, p.tokens);
    const uint32_t none = static_cast<uint32_t>(p.vocab);
    const T* dout = static_cast<const T*>(p.dout);
    float* mine = part + (c * 2) * p.dim + e0;

    uint32_t cur = key[MSEL_IDX(i0, p.tokens)];
    bool head = i0 > 0 && key[i0 - 1] == cur;  // the run began in an earlier chunk
    float acc[VE] = {};
    const auto store_part = [&](float* q) {
#pragma unroll
        for (int k = 0; k < VE; ++k)
            if (k < left) q[k] = acc[k];
    };
    for (int64_t i = i0; i < i1; i += kSegBatch) {
        uint32_t kk[kSegBatch];
        RawVec<T, VE> r[kSegBatch];
#pragma unroll
        for (int j = 0; j < kSegBatch; ++j) {
            const int64_t e = min(i + j, i1 - 1);
            kk[j] = i + j < i1 ? key[MSEL_IDX(e, p.tokens)] : none;
            const int64_t t = MSEL_IDX(static_cast<int64_t>(pos[e]), p.tokens);
            r[j] = ld_part<T, VE>(dout + t * p.dim + e0, left);
        }
#pragma unroll
        for (int j = 0; j < kSegBatch; ++j) {
            if (i + j >= i1) break;
            if (kk[j] != cur) {  // team-uniform
                if (cur != none) {
                    if (head) store_part(mine);
                    else write_row(p, cur, e0, left, acc, VE);
                }
                head = false;
                cur = kk[j];
#pragma unroll
                for (int k = 0; k < VE; ++k) acc[k] = 0.0f;
            }
            float v[VE];
            to_f32<T, VE>(r[j], v);
#pragma unroll
            for (int k = 0; k < VE; ++k) acc[k] += v[k];
        }
    }
    if (cur == none) return;
    const bool goes_on = i1 < p.tokens && key[i1] == cur;
    if (head) store_part(mine);
    else if (goes_on) store_part(mine + p.dim);
    else write_row(p, cur, e0, left, acc, VE);
}

// The runs that cross chunks: the chunk a run starts in adds the run's partial sums, row lanes
// of the block every RL-th each, then the row lanes in order.
__global__ __launch_bounds__(256) void embed_join_kernel(EmbedParams p, EmbedPlan pl, int S,
                                                         int nvec) {
    __shared__ float red[256][4];
    const char* ws = static_cast<const char*>(p.ws);
    const uint32_t* key = reinterpret_cast<const uint32_t*>(ws + pl.key[(pl.passes - 1) & 1]);
    const float* part = reinterpret_cast<const float*>(ws + pl.partial);
    const int64_t c = blockIdx.x;  // c + 1 < nseg
    const uint32_t k = key[(c + 1) * kSeg - 1];
    if (k == static_cast<uint32_t>(p.vocab) || key[(c + 1) * kSeg] != k) return;
    if (key[c * kSeg] == k && c > 0 && key[c * kSeg - 1] == k) return;  // began before
    int64_t lo = c + 1, hi = pl.nseg - 1;  // the last chunk whose first entry is in the run
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        if (key[MSEL_IDX(mid * kSeg, p.tokens)] == k) lo = mid;
        else hi = mid - 1;
    }
    const int rl = threadIdx.x / S, lane = threadIdx.x % S, RL = 256 / S;
    const int cv = blockIdx.y * S + lane;
    const int e0 = cv * 4, left = cv < nvec ? p.dim - e0 : 0;
    float acc[4] = {};
    const int64_t n = lo - c + 1;
#pragma unroll 4
    for (int64_t j = rl; j < n; j += RL) {
        // row 0 is the run's part in its first chunk, the others the heads of the next ones
        const int64_t row = j == 0 ? c * 2 + 1 : (c + j) * 2;
        float v[4];
        to_f32<float, 4>(ld_part<float, 4>(
                             part + MSEL_IDX(row, static_cast<int64_t>(pl.nseg) * 2) * p.dim + e0,
                             left), v);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] += v[q];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) red[threadIdx.x][q] = acc[q];
    __syncthreads();
    if (rl != 0 || left <= 0) return;
    for (int r = 1; r < RL; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] += red[r * S + lane][q];
    write_row(p, k, e0, left, acc, 4);
}

int team_of(int nvec, int most) {
    int s = 8;
    while (s < nvec && s < most) s *= 2;
    return s;
}

template <typename T, typename TW, int VE>
hipError_t embed_fwd_go(const EmbedParams& p, hipStream_t stream) {
    const int nvec = (p.dim + VE - 1) / VE;
    const int block_tokens = std::max(1, 1024 / nvec);
    const int64_t blocks = (p.tokens + block_tokens - 1) / block_tokens;
    hipLaunchKernelGGL((embed_fwd_kernel<T, TW, VE>), dim3(static_cast<unsigned>(blocks)),
                       dim3(256), 0, stream, p, nvec, make_fastdiv(static_cast<uint32_t>(nvec)),
                       block_tokens);
    return hipGetLastError();
}

}  // namespace

size_t embed_workspace_bytes(int64_t tokens, int vocab, int dim) {
    return embed_plan(tokens, vocab, dim).bytes;
}

hipError_t launch_embed_fwd(const EmbedParams& p, bool wbf16, bool bf16, hipStream_t stream) {
    if (bf16)
        return wbf16 ? embed_fwd_go<bf16_t, bf16_t, 8>(p, stream)
                     : embed_fwd_go<bf16_t, float, 8>(p, stream);
    return wbf16 ? embed_fwd_go<float, bf16_t, 4>(p, stream)
                 : embed_fwd_go<float, float, 4>(p, stream);
}

hipError_t launch_embed_bwd(const EmbedParams& p, bool bf16, hipStream_t stream) {
    const EmbedPlan pl = embed_plan(p.tokens, p.vocab, p.dim);
    int fill = 0;
    if (p.base != p.dw) {
        const int64_t nv = static_cast<int64_t>(p.vocab) * p.dim / 4 / (pl.passes + 1);
        fill = static_cast<int>(std::clamp<int64_t>((nv + kSortThreads - 1) / kSortThreads, 1,
                                                    kFillBlocks));
    }
    const dim3 grid(static_cast<unsigned>(pl.nblocks + fill));
    hipLaunchKernelGGL(embed_count_kernel, grid, dim3(kSortThreads), 0, stream, p, pl);
    for (int pass = 0; pass < pl.passes; ++pass)
        hipLaunchKernelGGL(embed_place_kernel, grid, dim3(kSortThreads), 0, stream, p, pl, pass);
    {
        const int ve = bf16 ? 8 : 4;
        const int nvec = (p.dim + ve - 1) / ve;
        const int S = team_of(nvec, 256);
        const dim3 g(static_cast<unsigned>((pl.nseg + 256 / S - 1) / (256 / S)),
                     static_cast<unsigned>((nvec + S - 1) / S));
        if (bf16)
            hipLaunchKernelGGL((embed_sum_kernel<bf16_t, 8>), g, dim3(256), 0, stream, p, pl, S,
                               nvec);
        else
            hipLaunchKernelGGL((embed_sum_kernel<float, 4>), g, dim3(256), 0, stream, p, pl, S,
                               nvec);
    }
    if (pl.nseg > 1) {
        const int nvec = (p.dim + 3) / 4;
        const int S = team_of(nvec, 64);
        const dim3 g(static_cast<unsigned>(pl.nseg - 1), static_cast<unsigned>((nvec + S - 1) / S));
        hipLaunchKernelGGL(embed_join_kernel, g, dim3(256), 0, stream, p, pl, S, nvec);
    }
    return hipGetLastError();
}

MSEL_BOUNDS_TAKER(take_bounds_embed)

}  // namespace msel
