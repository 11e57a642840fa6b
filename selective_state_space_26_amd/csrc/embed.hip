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
//     a wavefront by ballots, so that the order is the tokens' own: deterministic.  Up to
//     kOneBlock tokens are sorted by one block in one launch, and up to kSelfCount by blocks that
//     each count all of them.  The sort needs few blocks and
//     waits on latency, so the same launches fill dw (with base or 0) on the remaining CUs;
//  2. segment sums: the sorted positions in chunks of `seg` entries; a team of lanes adds its
//     chunk's rows in fp32.  An id's run inside a chunk is written to dw directly; a run that
//     crosses chunks leaves one partial sum per chunk;
//  3. the partial sums of each crossing run are added in chunk order.
// No floating-point atomics.  The segment sums take the same time whatever the ids; a run is
// joined by one block per slab of columns, so a batch of mostly one id takes longer (2^18 x 64 fp32
// of 16 ids 32 us, of one id 80).  (Counting a pass's digits with global atomics in the pass before
// saved a launch and cost 22 us: the most frequent ids' counters are one address each.)
// Measured: lookup of 16384 x 768, fp32 to bf16, 10 us (44 MB); gradient of 16384 bf16 rows of 50257
// ids 53 to 60 us: 8 + 10 + 8 + 10 for the sort's launches, which the fill of 154 MB bounds, 12 for
// the segment sums, 7 for the join; of 262144 fp32 rows of 64 for 16 ids 3 + 7, 14 and 9.
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
// Blocks of the sort: every one reads all blocks' counts, so fewer where there are many digits
// (2^18 tokens of 17 ids: 36.2 us with 128 blocks, 34.8 with 256).
constexpr int max_sort_blocks(int dbits) { return dbits <= 6 ? 256 : 128; }
// Up to so many tokens every sort block counts all of them itself, which saves a launch per pass:
// 8192 tokens of 50257 ids 41 us with it, 49 without; 32768 of 200 ids 33 and 26.
constexpr int64_t kSelfCount = 8192;
constexpr int kOneBlock = 2048;  // tokens that one block sorts alone
constexpr int kFillBlocks = 512;
constexpr int kSegBatch = 8;     // rows of a chunk in flight at a time
constexpr int kJoinThreads = 256;
// Partial sums of a run in flight per lane: 2^18 x 768 fp32 of one id 530 us with 8, 440 with 16.
constexpr int kJoinBatch = 16;
constexpr int kJoinBlocks = 1024;  // blocks per slab of columns that look for runs to join

struct EmbedPlan {
    int passes, dbits, nblocks;
    int chunk;       // tokens per sort block
    int seg, nseg;   // sorted entries per segment-sum chunk, chunks
    bool self;       // every block counts all tokens' digits itself
    int launches;    // of the sort, each with a share of the fill
    size_t key[2], pos[2], table, partial, bytes;  // offsets into the workspace
};

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

int team_of(int nvec, int most) {
    int s = 8;
    while (s < nvec && s < most) s *= 2;
    return s;
}

EmbedPlan embed_plan(int64_t tokens, int vocab, int dim) {
    EmbedPlan pl{};
    int bits = 1;
    while ((int64_t(1) << bits) <= vocab) ++bits;  // the sentinel is vocab itself
    pl.passes = (bits + kDigitBits - 1) / kDigitBits;
    pl.dbits = (bits + pl.passes - 1) / pl.passes;
    const int64_t tiles = (tokens + kSortThreads - 1) / kSortThreads;
    const int64_t blocks =
        tokens <= kOneBlock ? 1 : std::min<int64_t>(max_sort_blocks(pl.dbits), tiles);
    pl.chunk = static_cast<int>((tiles + blocks - 1) / blocks * kSortThreads);
    pl.nblocks = static_cast<int>((tokens + pl.chunk - 1) / pl.chunk);
    pl.self = pl.nblocks > 1 && tokens <= kSelfCount;
    pl.launches = pl.nblocks == 1 ? 1 : pl.self ? pl.passes : 2 * pl.passes;
    // short chunks while the teams would not fill the chip (a chunk is a team's work), long ones
    // for many rows, which leave fewer partial sums: 2048 x 1024 of 32000 ids took 32 us with 8
    // entries and 40 with 32, 262144 x 64 of 16 ids 48 and 36, 16384 x 768 of 50257 ids 53 with 16
    const int64_t lanes = tokens * std::min(256, (dim + 7) / 8);
    pl.seg = 8;
    while (pl.seg < 32 && lanes / pl.seg > 98304) pl.seg *= 2;
    pl.nseg = static_cast<int>((tokens + pl.seg - 1) / pl.seg);
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
    pl.table = take(static_cast<size_t>(kBins) * pl.nblocks * 4);
    pl.partial = take(static_cast<size_t>(pl.nseg) * 2 * dim * 4);
    pl.bytes = at;
    return pl;
}

template <typename T, typename TW, int VE>
__global__ __launch_bounds__(256) void embed_fwd_kernel(EmbedParams p, int nvec, FastDiv by_nvec,
                                                        int block_tokens) {
    const int64_t t0 =
        (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * block_tokens;
    if (t0 >= p.tokens) return;
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

__device__ __forceinline__ uint32_t* part_of(const EmbedParams& p, size_t offset) {
    return reinterpret_cast<uint32_t*>(static_cast<char*>(p.ws) + offset);
}

// (key, position) of entry t before pass `pass`.
__device__ __forceinline__ uint32_t key_at(const EmbedParams& p, const EmbedPlan& pl, int pass,
                                           int64_t t) {
    return pass == 0 ? key_of(p, t) : part_of(p, pl.key[(pass + 1) & 1])[MSEL_IDX(t, p.tokens)];
}

// Counts the digits of pass `pass` in this block's tokens into cnt[1 << dbits] (LDS).
__device__ __forceinline__ void count_digits(const EmbedParams& p, const EmbedPlan& pl, int pass,
                                             uint32_t* cnt) {
    const int nb = 1 << pl.dbits;
    for (int i = threadIdx.x; i < nb; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * pl.chunk;
    const int64_t t1 = min(t0 + pl.chunk, p.tokens);
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kSortThreads)
        atomicAdd(&cnt[(key_at(p, pl, pass, t) >> (pass * pl.dbits)) & (nb - 1)], 1u);
    __syncthreads();
}

// Digit counts per block of one pass: table[block][digit].
__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(EmbedParams p, EmbedPlan pl,
                                                                   int pass) {
    __shared__ uint32_t cnt[kBins];
    if (static_cast<int>(blockIdx.x) >= pl.nblocks) {
        fill_share(p, 2 * pass, pl.launches, blockIdx.x - pl.nblocks, gridDim.x - pl.nblocks);
        return;
    }
    count_digits(p, pl, pass, cnt);
    const int nb = 1 << pl.dbits;
    uint32_t* table = part_of(p, pl.table);
    for (int d = threadIdx.x; d < nb; d += kSortThreads)
        table[MSEL_IDX(static_cast<int>(blockIdx.x) * nb + d, kBins * pl.nblocks)] = cnt[d];
}

// Where a placing block has the counts from: a block alone counts its tokens and makes all passes,
// of several each counts all tokens itself, or reads the counts of the launch before.
enum class Counts { kAlone, kSelf, kTable };

// Places the tokens of pass `pass` in digit order (stable).
template <Counts FROM>
__global__ __launch_bounds__(kSortThreads) void embed_place_kernel(EmbedParams p, EmbedPlan pl,
                                                                   int pass) {
    __shared__ uint32_t run[kBins];  // next free place of each digit
    __shared__ uint32_t cnt[kSortWaves][kBins];
    __shared__ uint32_t wsum[kSortWaves];
    constexpr bool alone = FROM == Counts::kAlone;
    if (static_cast<int>(blockIdx.x) >= pl.nblocks) {
        fill_share(p, alone ? 0 : FROM == Counts::kSelf ? pass : 2 * pass + 1, pl.launches,
                   blockIdx.x - pl.nblocks, gridDim.x - pl.nblocks);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nb = 1 << pl.dbits;
    const uint32_t mask = static_cast<uint32_t>(nb) - 1u;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * pl.chunk;
    const int64_t t1 = min(t0 + pl.chunk, p.tokens);
    do {
        // where this block's tokens of each digit go: all smaller digits, then this digit in the
        // blocks before
        uint32_t total = 0, before = 0;
        if constexpr (alone) {
            count_digits(p, pl, pass, &cnt[0][0]);
            if (tid < nb) total = cnt[0][tid];
            __syncthreads();
        } else if constexpr (FROM == Counts::kSelf) {
            // the tokens before this block's in rows 0..7 of cnt, the others in 8..15, two
            // wavefronts a row
            for (int i = tid; i < kSortWaves * nb; i += kSortThreads)
                cnt[i >> pl.dbits][i & (nb - 1)] = 0;
            __syncthreads();
            const int shift = pass * pl.dbits;
#pragma unroll 8
            for (int64_t t = tid; t < p.tokens; t += kSortThreads)
                atomicAdd(
                    &cnt[(wave & 7) + (t < t0 ? 0 : 8)][(key_at(p, pl, pass, t) >> shift) & mask],
                    1u);
            __syncthreads();
            if (tid < nb)
#pragma unroll
                for (int w = 0; w < kSortWaves; ++w) {
                    total += cnt[w][tid];
                    before += w < kSortWaves / 2 ? cnt[w][tid] : 0u;
                }
            __syncthreads();
        } else {
            const uint32_t* table = part_of(p, pl.table);
            const int d = tid & (nb - 1), grp = tid >> pl.dbits, grps = kSortThreads >> pl.dbits;
            const int me = static_cast<int>(blockIdx.x);
#pragma unroll 8
            for (int j = grp; j < pl.nblocks; j += grps) {
                const uint32_t c = table[MSEL_IDX(j * nb + d, kBins * pl.nblocks)];
                total += c;
                before += j < me ? c : 0u;
            }
            // the groups' sums, [2][grps][nb] in cnt
            uint32_t* sums = &cnt[0][0];
            sums[tid] = total;
            sums[kSortThreads + tid] = before;
            __syncthreads();
            total = before = 0;
            if (tid < nb)
                for (int g = 0; g < grps; ++g) {
                    total += sums[g * nb + tid];
                    before += sums[kSortThreads + g * nb + tid];
                }
            __syncthreads();
        }
        // exclusive sums of the totals over the digits (0 in threads past them)
        uint32_t incl = total;
#pragma unroll
        for (int s = 1; s < 64; s *= 2) {
            const uint32_t v = __shfl_up(incl, s);
            incl += lane >= s ? v : 0u;
        }
        if (lane == 63) wsum[wave] = incl;
        __syncthreads();
        uint32_t base = 0;
        for (int w = 0; w < wave; ++w) base += wsum[w];
        if (tid < nb) run[tid] = base + incl - total + before;

        uint32_t* key_out = part_of(p, pl.key[pass & 1]);
        uint32_t* pos_out = part_of(p, pl.pos[pass & 1]);
        const int shift = pass * pl.dbits;
        for (int64_t tb = t0; tb < t1; tb += kSortThreads) {  // block-uniform
            for (int i = tid; i < kSortWaves * nb; i += kSortThreads)
                cnt[i >> pl.dbits][i & (nb - 1)] = 0;
            __syncthreads();
            const int64_t t = tb + tid;
            const bool in = t < t1;
            uint32_t key = 0, pos = 0;
            if (in) {
                key = key_at(p, pl, pass, t);
                pos = pass == 0 ? static_cast<uint32_t>(t)
                                : part_of(p, pl.pos[(pass + 1) & 1])[MSEL_IDX(t, p.tokens)];
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
            if (tid < nb) {
                uint32_t s = run[tid];
#pragma unroll
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
            }
            __syncthreads();
        }
        // a block alone goes on: its own writes are visible to it after the barrier
    } while (alone && ++pass < pl.passes);
}

template <int VE>
__device__ __forceinline__ void write_row(const EmbedParams& p, uint32_t v, int e0, int left,
                                          const float (&acc)[VE]) {
    const int64_t at = static_cast<int64_t>(MSEL_IDX(v, p.vocab)) * p.dim + e0;
    float o[VE] = {};
    if (p.base != nullptr) to_f32<float, VE>(ld_part<float, VE>(p.base + at, left), o);
#pragma unroll
    for (int k = 0; k < VE; ++k) o[k] = fmaf(p.scale, acc[k], o[k]);
    st_part<float, VE>(p.dw + at, from_f32<float, VE>(o), left);
}

// Segment sums: a team of S lanes (S vectors of a row) per chunk of pl.seg sorted entries.  The
// chunk's ids and positions are loaded by the team's lanes, R = min(S, 64) at a time, and handed
// round the wavefront.
template <typename T, int VE>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedParams p, EmbedPlan pl, int S,
                                                        int nvec) {
    const uint32_t* key = part_of(p, pl.key[(pl.passes - 1) & 1]);
    const uint32_t* pos = part_of(p, pl.pos[(pl.passes - 1) & 1]);
    const int team = threadIdx.x / S, lane = threadIdx.x % S;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * (256 / S) + team;
    const bool on = c < pl.nseg;  // team-uniform; idle teams keep their lanes for the handing round
    const int cv = blockIdx.y * S + lane;
    const int e0 = cv * VE, left = on && cv < nvec ? p.dim - e0 : 0;
    const int64_t i0 = on ? c * pl.seg : 0;
    const int n = on ? static_cast<int>(min(static_cast<int64_t>(pl.seg), p.tokens - i0)) : 0;
    const uint32_t none = static_cast<uint32_t>(p.vocab);
    const T* dout = static_cast<const T*>(p.dout) + e0;
    float* mine = reinterpret_cast<float*>(part_of(p, pl.partial)) + (c * 2) * p.dim + e0;
    const int R = min(S, 64), rl = lane & (R - 1), first = lane_id() - rl;

    // the ids before and after the chunk: a run may begin before it, or go on after it
    const uint32_t before = i0 > 0 ? key[i0 - 1] : none;
    const uint32_t after = i0 + n < p.tokens ? key[i0 + n] : none;
    uint32_t mk = rl < n ? key[i0 + rl] : none;
    uint32_t mp = rl < n ? pos[i0 + rl] : 0u;
    uint32_t cur = __shfl(mk, first);
    bool head = i0 > 0 && before == cur;
    float acc[VE] = {};
    for (int r = 0; r < pl.seg; r += R) {  // block-uniform
        const uint32_t ks = mk, ps = mp;
        if (r + R < pl.seg) {  // the next ids while these rows are added
            const int j = r + R + rl;
            mk = j < n ? key[i0 + j] : none;
            mp = j < n ? pos[i0 + j] : 0u;
        }
        const int rows = min(R, pl.seg - r);
        for (int j0 = 0; j0 < rows; j0 += kSegBatch) {
            uint32_t kk[kSegBatch];
            RawVec<T, VE> v[kSegBatch];
#pragma unroll
            for (int j = 0; j < kSegBatch; ++j) {
                kk[j] = __shfl(ks, first + j0 + j);
                const int64_t t = MSEL_IDX(static_cast<int64_t>(__shfl(ps, first + j0 + j)), p.tokens);
                v[j].w = 0;
                if (left > 0 && kk[j] != none) v[j] = ld_part<T, VE>(dout + t * p.dim, left);
            }
#pragma unroll
            for (int j = 0; j < kSegBatch; ++j) {
                if (r + j0 + j >= n) break;  // team-uniform
                if (kk[j] != cur) {
                    if (cur != none && left > 0) {
                        if (head) st_part<float, VE>(mine, from_f32<float, VE>(acc), left);
                        else write_row<VE>(p, cur, e0, left, acc);
                    }
                    head = false;
                    cur = kk[j];
#pragma unroll
                    for (int k = 0; k < VE; ++k) acc[k] = 0.0f;
                }
                float f[VE];
                to_f32<T, VE>(v[j], f);
#pragma unroll
                for (int k = 0; k < VE; ++k) acc[k] += f[k];
            }
        }
    }
    if (cur == none || left <= 0) return;
    if (head) st_part<float, VE>(mine, from_f32<float, VE>(acc), left);
    else if (after == cur) st_part<float, VE>(mine + p.dim, from_f32<float, VE>(acc), left);
    else write_row<VE>(p, cur, e0, left, acc);
}

// The runs that cross chunks: for each of the block's `look` (up to 64 at a time) chunks that such
// a run starts in, the block adds the run's partial sums, its row lanes every RL-th row each, then
// the row lanes in order.  A run of m tokens has m / seg partial sums, and a lane may add thousands
// of them one after another: a batch in a tree in fp32, the batches in fp64 (with fp32 alone the
// gradient of 2^18 equal rows of one id was off by 500 x 2^-24 of itself).
__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(EmbedParams p, EmbedPlan pl,
                                                                  int S, int nvec, int look) {
    __shared__ double red[4][kJoinThreads];
    const uint32_t* key = part_of(p, pl.key[(pl.passes - 1) & 1]);
    const float* part = reinterpret_cast<const float*>(part_of(p, pl.partial));
    const int64_t seg = pl.seg;
    const uint32_t none = static_cast<uint32_t>(p.vocab);
    const int rl = threadIdx.x / S, lane = threadIdx.x % S, RL = kJoinThreads / S;
    const int cv = blockIdx.y * S + lane;
    const int e0 = cv * 4, left = cv < nvec ? p.dim - e0 : 0;
    for (int l0 = 0; l0 < look; l0 += 64) {
        const int64_t cb = static_cast<int64_t>(blockIdx.x) * look + l0;
        bool starts = false;
        if (lane_id() < look - l0 && cb + lane_id() + 1 < pl.nseg) {
            const int64_t c = cb + lane_id();
            const uint32_t k = key[(c + 1) * seg - 1], next = key[(c + 1) * seg], first = key[c * seg];
            const uint32_t prev = c > 0 ? key[c * seg - 1] : none;
            starts = k != none && next == k && !(first == k && prev == k);
        }
        uint64_t todo = __ballot(starts);  // the same in every wavefront
        for (; todo != 0; todo &= todo - 1) {  // block-uniform
            const int64_t c = cb + __builtin_ctzll(todo);
            const uint32_t k = key[(c + 1) * seg];
            // n: the chunks from c on whose first entries are in the run (but c's own), 64 at a
            // time: in strides of 1, 64, .. until one stride reaches past the run, then back
            const auto matches = [&](int64_t from, int64_t stride) {
                const int64_t j = from + lane_id() * stride;
                const bool in = j < pl.nseg && key[MSEL_IDX(j * seg, p.tokens)] == k;
                return __popcll(__ballot(in));  // ids are sorted: a prefix of the lanes
            };
            int64_t at = c + 1, stride = 1;
            int m = matches(at, 1);
            while (m == 64 && stride < pl.nseg) m = matches(at, stride *= 64);
            for (; stride > 1; m = matches(at, stride)) {
                at += (m - 1) * stride;
                stride /= 64;
            }
            const int64_t n = at + m - c;
            // row 0 is the run's part in its first chunk, the others the heads of the next ones
            const auto part_row = [&](int64_t j) {
                RawVec<float, 4> v;
                v.w = 0;
                const int64_t row = j == 0 ? c * 2 + 1 : (c + j) * 2;
                if (j < n)
                    v = ld_part<float, 4>(
                        part + MSEL_IDX(row, static_cast<int64_t>(pl.nseg) * 2) * p.dim + e0, left);
                return v;
            };
            float s[kJoinBatch][4];
            double acc[4] = {};
            if (n <= RL) {  // block-uniform: most runs, one row per row lane
                to_f32<float, 4>(part_row(rl), s[0]);
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[q] = static_cast<double>(s[0][q]);
            } else {
                for (int64_t j0 = rl; j0 < n; j0 += kJoinBatch * RL) {
#pragma unroll
                    for (int i = 0; i < kJoinBatch; ++i)
                        to_f32<float, 4>(part_row(j0 + i * RL), s[i]);
#pragma unroll
                    for (int h = kJoinBatch / 2; h > 0; h /= 2)
#pragma unroll
                        for (int i = 0; i < h; ++i)
#pragma unroll
                            for (int q = 0; q < 4; ++q) s[i][q] += s[i + h][q];
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[q] += static_cast<double>(s[0][q]);
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) red[q][threadIdx.x] = acc[q];
            __syncthreads();
            if (rl == 0 && left > 0) {
                const int rows = static_cast<int>(min(static_cast<int64_t>(RL), n));
                for (int r = 1; r < rows; ++r)
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[q] += red[q][r * S + lane];
                float sum[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) sum[q] = static_cast<float>(acc[q]);
                write_row<4>(p, k, e0, left, sum);
            }
            __syncthreads();  // red is free again
        }
    }
}

template <typename T, typename TW, int VE>
hipError_t embed_fwd_go(const EmbedParams& p, hipStream_t stream) {
    const int nvec = (p.dim + VE - 1) / VE;
    const int block_tokens = std::max(1, 1024 / nvec);
    const int64_t blocks = (p.tokens + block_tokens - 1) / block_tokens;
    const int64_t most = 1 << 23;  // a grid's dimension has fewer than 2^32 threads
    const dim3 grid(static_cast<unsigned>(std::min(blocks, most)),
                    static_cast<unsigned>((blocks + most - 1) / most));
    hipLaunchKernelGGL((embed_fwd_kernel<T, TW, VE>), grid, dim3(256), 0, stream, p, nvec,
                       make_fastdiv(static_cast<uint32_t>(nvec)), block_tokens);
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
        const int64_t nv = static_cast<int64_t>(p.vocab) * p.dim / 4 / pl.launches;
        fill = static_cast<int>(std::clamp<int64_t>((nv + kSortThreads - 1) / kSortThreads, 1,
                                                    kFillBlocks));
    }
    const dim3 grid(static_cast<unsigned>(pl.nblocks + fill));
    const auto place = [&](auto kernel, int pass) {
        hipLaunchKernelGGL(kernel, grid, dim3(kSortThreads), 0, stream, p, pl, pass);
    };
    if (pl.nblocks == 1) {
        place(embed_place_kernel<Counts::kAlone>, 0);
    } else {
        for (int pass = 0; pass < pl.passes; ++pass) {
            if (pl.self) {
                place(embed_place_kernel<Counts::kSelf>, pass);
            } else {
                place(embed_count_kernel, pass);
                place(embed_place_kernel<Counts::kTable>, pass);
            }
        }
    }
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
        const int look = std::max(4, (pl.nseg - 1 + kJoinBlocks - 1) / kJoinBlocks);
        const dim3 g(static_cast<unsigned>((pl.nseg - 1 + look - 1) / look),
                     static_cast<unsigned>((nvec + S - 1) / S));
        hipLaunchKernelGGL(embed_join_kernel, g, dim3(kJoinThreads), 0, stream, p, pl, S, nvec,
                           look);
    }
    return hipGetLastError();
}

MSEL_BOUNDS_TAKER(take_bounds_embed)

}  // namespace msel
