// gated_mlp.hip -- the gated feed-forward block out = act(x Wg^T) * (x Wu^T) and its backward
//   dG = dout U act'(G), dU = dout act(G);  dx = dG Wg + dU Wu;  dWg = dG^T x, dWu = dU^T x
// as MFMA products of rows with consecutive k: C[m][n] = sum_k A[m][k] B[n][k].
//
// The matrix cores bound it.  A block computes a tile of C with both operands staged in LDS, two
// stages of 128 bytes of k in turn, loaded without a register between (global_load_lds).  A step's
// fragments are read from LDS during the MFMAs of the step before, across the stages' borders too:
// a stage's place is loaded again as soon as its last fragments have been read, before they are
// used.  A row of a stage is 8 chunks of 16 bytes, chunk c of row r at place c ^ (r / 2 & 7): the
// 16 lanes that LDS serves together read one chunk of 16 rows, which then cover all 64 banks.  The
// result goes out through LDS too, in whole rows of the tile.  In the fused product the B rows of a
// wavefront are 32 rows of Wg and the same 32 of Wu, so that a lane holds G and U of the same
// elements and the activation and the product need no exchange. The MFMA's rows are C's columns, so
// that a lane holds consecutive columns of a row of C.  The backward's products over the hidden
// width and over the tokens read their operands by rows of k, as they lie in memory; LDS turns them
// (the transposing reads of gfx950), and their bf16 stages come through registers.
//
// Operands whose rows are no multiple of 16 bytes, or below a stage, are copied into padded rows
// first.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block_kernels.hpp"
#include "lm_device.hpp"

namespace msel {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kStageBytes = 128;  // of k per stage
constexpr int kRing = 2;          // stages in LDS
constexpr int kSteps = kStageBytes / 32;
// fp32: stages whose products are summed before their sum is added to another.  An MFMA adds 2
// products and rounds, and a row of 2048 such steps was off by up to 2.4 times as much as parts of
// 256 are (2 tokens of 1998: 1.1e-6 of the result).  They cost 0.5% of a product's time.  Tiles of
// 256 x 256 have no registers for a second sum: the plan takes them only where no block sums more
// stages than these (2048 x 4096 -> 8192, forward: 10 u of the result with 128 x 128 and 2080 us,
// 29 u and 2016 us with 256 x 256 before; 16384 x 512 -> 1024: 268 us with 256 x 256, 280).
constexpr int kPartStages = 16;

template <typename T>
constexpr int kStageK = kStageBytes / static_cast<int>(sizeof(T));

// acc += a b^T over 32 bytes of k: 16 bytes per lane of a row each, the lower half of the lanes the
// first 16, the upper half the others.
__device__ __forceinline__ void mfma_step(const bf16_t*, const u32x4& a, const u32x4& b,
                                          f32x16& acc) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}
__device__ __forceinline__ void mfma_step(const float*, const u32x4& a, const u32x4& b,
                                          f32x16& acc) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]), __uint_as_float(b[e]),
                                                   acc, 0, 0, 0);
}

// act(z) and its derivative.  gelu in its tanh form is z s, s = sigmoid(2 c (z + 0.044715 z^3)).
constexpr float kTwoC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
template <bool GELU>
__device__ __forceinline__ float act_of(float z) {
    return z * sigmoid_f(GELU ? kTwoC * z * fmaf(0.044715f * z, z, 1.0f) : z);
}
template <bool GELU>
__device__ __forceinline__ void act_grad(float z, float& v, float& slope) {
    const float s = sigmoid_f(GELU ? kTwoC * z * fmaf(0.044715f * z, z, 1.0f) : z);
    v = z * s;
    const float w = v - v * s;
    // w is 0 long before the polynomial beside it leaves fp32's range
    slope = GELU ? fmaf(w, kTwoC * fminf(fmaf(0.134145f * z, z, 1.0f), 1e30f), s) : w + s;
}
// What a value's rounding to bf16 leaves: nothing where it became an infinity or a NaN, which stand
// for the value alone.
__device__ __forceinline__ float rest_of(float v) {
    const float rounded = bf16lo(pack_bf16(v, 0.0f));
    return fabsf(rounded) < INFINITY ? v - rounded : 0.0f;
}
// f(GELU as a type): one branch around a whole epilogue, not two activations per element.
template <typename Fn>
__device__ __forceinline__ void with_act(int gelu, Fn f) {
    if (gelu)
        f(std::true_type());
    else
        f(std::false_type());
}

// What a product is, which also says how its operands lie: with consecutive k (rows of A and B), or
// by rows of k (columns of A and B are consecutive).
enum class Kind {
    kGate,      // out = act(G) * U: A = x, B = Wg and Wu, all with consecutive k
    kGateGrad,  // dG and dU from G, U and dout: the same
    kInput,     // dx = dG Wg + dU Wu: A = (dG, dU) with consecutive k, B = Wg, then Wu by rows of k
    kWeights,   // dW = (dG, dU)^T x: both by rows of k, the tokens
};
constexpr bool dual(Kind k) { return k == Kind::kGate || k == Kind::kGateGrad; }

struct ProductParams {
    int64_t M;       // rows of C
    int N;           // columns of C; in the fused products the hidden width
    int64_t K;       // along k: elements of a row, or rows (of each part of B)
    const void* a;
    const void* b0;
    const void* b1;  // the other weight
    int64_t lda, ldb;
    int64_t wa, wb;  // elements of a row of A and B that may be read, where they lie by rows of k
    int stages, half;  // stages in all, and of one part: B0, B1, then both with the low parts of A
    int64_t low;       // kWeights: elements from A to its low parts
    int splits, per_split;  // blocks that share a tile's stages, and stages of each
    void* c0;        // rows [0, rows0) of C
    void* c1;        // rows from `split` on; those between go nowhere
    int64_t rows0, split, ldc;
    float* part;       // not null: C goes there, [splits][M][N], or G and U, [splits][2][M][N]
    const void* dout;  // kGateGrad: [M, N]
    int hp;            // kGateGrad: dG in columns [0, hp) of C, dU in [hp, 2 hp)
    int with_low;      // kGateGrad: what their rounding left in [2 hp, 4 hp)
    int gelu;
    int tm, tn;        // tiles
};

// The tile of a block and its part of the stages: consecutive tiles on one XCD, in bands of 8 tiles
// of rows, so that the blocks that run together share rows of both operands in its L2 (in a grid
// that gives each part to all XCDs, 61% of the L2's reads missed).
__device__ __forceinline__ bool tile_at(const ProductParams& p, int& m, int& n, int& part) {
    const int64_t tiles = static_cast<int64_t>(p.tm) * p.tn, all = tiles * p.splits;
    const int64_t bid = blockIdx.y * static_cast<int64_t>(gridDim.x) + blockIdx.x;
    if (bid >= all) return false;
    const int64_t at = gridDim.y == 1 ? xcd_order(blockIdx.x, gridDim.x) : bid;
    part = p.splits == 1 ? 0 : static_cast<int>(at / tiles);
    const int id = static_cast<int>(at - part * tiles);
    constexpr int kBand = 8;
    const int width = kBand * p.tn;
    const int band = id / width, in = id - band * width;
    const int rows = min(kBand, p.tm - band * kBand);
    m = band * kBand + in % rows;
    n = in / rows;
    return true;
}

typedef __attribute__((address_space(1))) const void GlobalVoid;
typedef __attribute__((address_space(3))) void LdsVoid;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 LdsS16x4;

// MFMA row i of a fragment of B is column order32(i) of its 32 columns of C: the result's rows
// 8 g + 4 h + e, which a lane of half h holds in order of g and e, are then 16 consecutive columns.
__device__ __forceinline__ int order32(int i) {
    return ((i >> 2) & 1) * 16 + (i >> 3) * 4 + (i & 3);
}

// An operand of W rows (or columns of C's side) per stage in LDS, by chunks of 16 bytes.
//
// Consecutive k: [W][8 chunks], chunk c of row r at place c ^ (r / 2 & 7): two rows are as long as
// the 64 banks, and the 16 lanes that LDS serves together read one chunk of 16 rows.  ORDER: rows
// in the order order32.
//
// By rows of k: [rows of k][W columns].  bf16 fragments are read with the transposing read, which
// gives each lane of 16 the 4 values of its column from 4 rows of 16 columns; two such groups read
// 64 bytes of 4 rows, which the swizzle puts in different quarters of the banks.  fp32 fragments
// are single values: 32 columns of rows k and k + 4, in different halves of the banks.
template <typename T, int W, bool BY_ROWS, bool ORDER>
struct Operand {
    static constexpr int kBytes = W * kStageBytes;
    static constexpr int kPerChunk = 16 / static_cast<int>(sizeof(T));
    static constexpr int kChunks = BY_ROWS ? W / kPerChunk : kStageBytes / 16;  // of a row in LDS

    __device__ __forceinline__ static int swizzle(int r) {
        if constexpr (!BY_ROWS) return (r >> 1) & 7;
        if constexpr (sizeof(T) == 4) return ((r >> 2) & 1) << 3;
        return kChunks == 8 ? ((r >> 1) & 1) << 2 : (r & 3) << 2;
    }
    // fragment f (32 rows) of step s: 16 bytes per lane
    __device__ __forceinline__ static u32x4 read(const char* at, int f, int s, int lane) {
        const int h = lane >> 5;
        if constexpr (!BY_ROWS) {
            const int r = f * 32 + (lane & 31);
            return *reinterpret_cast<const u32x4*>(at + r * kStageBytes +
                                                   (((2 * s + h) ^ swizzle(lane)) * 16));
        } else if constexpr (sizeof(T) == 4) {
            const int c = f * 32 + (ORDER ? order32(lane & 31) : lane & 31);
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 8 * s + 4 * h + e;
                const int chunk = (c >> 2) ^ swizzle(k);
                v[e] = *reinterpret_cast<const uint32_t*>(at + k * (W * 4) + chunk * 16 +
                                                          (c & 3) * 4);
            }
            return v;
        } else {
            const int q = (lane >> 4) & 1, t = lane & 15, seg = t & 3;
            // where the 4 columns lie that this lane's address stands for
            const int c = f * 32 + (ORDER ? 16 * (seg & 1) + 4 * (2 * q + (seg >> 1))
                                          : 16 * q + 4 * seg);
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = 16 * s + 8 * h + 4 * e + (t >> 2);
                const int chunk = (c >> 3) ^ swizzle(k);
                const s16x4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (LdsS16x4*)(at + k * (W * 2) + chunk * 16 + (c & 4) * 2));
                typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                const u32x2 u = __builtin_bit_cast(u32x2, w);
                v[2 * e] = u[0];
                v[2 * e + 1] = u[1];
            }
            return v;
        }
    }
};

// A tile of C on its way out: BM rows of W columns of type U in LDS, in chunks of 16 bytes,
// swizzled so that 16 rows of one chunk (a wavefront writes them) and a row's chunks (it reads
// them) both cover all banks.
template <typename U, int W>
struct OutTile {
    static constexpr int kPerChunk = 16 / static_cast<int>(sizeof(U));
    static constexpr int kChunks = W / kPerChunk;
    static_assert(kChunks == 8 || kChunks % 16 == 0, "the swizzle stays inside a row");
    __device__ __forceinline__ static int place(int r, int c) {
        return (r * kChunks + (c ^ (kChunks == 8 ? (r >> 1) & 7 : r & 15))) * 16;
    }
    // 16 columns from `col` on of row r
    __device__ __forceinline__ static void put(char* lds, int r, int col, const float (&v)[16]) {
#pragma unroll
        for (int q = 0; q < 16 / kPerChunk; ++q) {
            float w[kPerChunk];
#pragma unroll
            for (int e = 0; e < kPerChunk; ++e) w[e] = v[q * kPerChunk + e];
            const RawVec<U, kPerChunk> raw = from_f32<U, kPerChunk>(w);
            __builtin_memcpy(lds + place(r, col / kPerChunk + q), &raw, 16);
        }
    }
    __device__ __forceinline__ static void get(const char* lds, int r, int col, float (&v)[16]) {
#pragma unroll
        for (int q = 0; q < 16 / kPerChunk; ++q) {
            RawVec<U, kPerChunk> raw;
            __builtin_memcpy(&raw, lds + place(r, col / kPerChunk + q), 16);
            float w[kPerChunk];
            to_f32<U, kPerChunk>(raw, w);
#pragma unroll
            for (int e = 0; e < kPerChunk; ++e) v[q * kPerChunk + e] = w[e];
        }
    }
};

// Up to a vector's columns of a row of n: columns [col, col + VE).
template <typename U, int VE>
__device__ __forceinline__ void store_columns(U* row, int col, int n, const RawVec<U, VE>& r) {
    if (col + VE <= n)
        st_raw<U, VE>(row + MSEL_SPAN(col, VE, n), r);
    else if (col < n)
        st_part<U, VE>(row + col, r, n - col);
}

// All but the n loads issued last have landed, here and in the other wavefronts, and what this one
// read from LDS has arrived.
template <int N>
__device__ __forceinline__ void barrier_after() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// What this wavefront wrote to LDS and read from it has arrived, and the others' has.
__device__ __forceinline__ void barrier_of_lds() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// WM x WN wavefronts, each MI x 2 MFMA tiles of 32 x 32: a block computes WM MI 32 rows by
// WN 64 columns (in the fused products WN 32 columns of both weights).
template <typename T, int WM, int WN, int MI, Kind KIND>
__global__ __launch_bounds__(WM* WN * 64, 2) void product_kernel(ProductParams p) {
    constexpr int kThreads = WM * WN * 64;
    constexpr int BM = WM * MI * 32, BN = WN * 64;
    constexpr bool kDual = dual(KIND);
    constexpr bool kRowsA = KIND == Kind::kWeights, kRowsB = !kDual;
    using OpA = Operand<T, BM, kRowsA, false>;
    using OpB = Operand<T, BN, kRowsB, true>;
    constexpr int LA = OpA::kBytes / 16 / kThreads, LB = OpB::kBytes / 16 / kThreads;
    constexpr int kStage = OpA::kBytes + OpB::kBytes;
    // bf16 operands by rows of k: the compiler lets no transposing read pass a load that goes to
    // LDS (each waited for all of them), so that such stages come through registers: dx of 16384 x
    // 768 -> 2048 145 us before, 116 so, the weights' gradients 136 and 112
    constexpr bool kHeld = sizeof(T) == 2 && !kDual;
    constexpr int CW = kDual ? BN / 2 : BN;  // columns of C
    static_assert(LA * kThreads * 16 == OpA::kBytes && LB * kThreads * 16 == OpB::kBytes,
                  "whole rounds");
    extern __shared__ __align__(16) char lds[];

    int tile_m, tile_n, split;
    if (!tile_at(p, tile_m, tile_n, split)) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = lane_id();
    const int wm = wave / WN, wn = wave % WN;
    const int64_t m0 = static_cast<int64_t>(tile_m) * BM;
    const int n0 = tile_n * (kDual ? BN / 2 : BN);

    // this thread's chunks of the first stage.  Rows and columns past the end repeat the last ones
    // (their results are not stored); rows of k past the end are zeroed in LDS.
    // By rows of k a thread's chunks are the same columns of rows kRoundA or kRoundB apart: one
    // address.
    constexpr int kRoundA = kThreads / OpA::kChunks, kRoundB = kThreads / OpB::kChunks;
    static_assert(kRoundA % 8 == 0 && kRoundB % 8 == 0, "the swizzle is that of the first row");
    constexpr int SA = kRowsA ? 1 : LA, SB = kRowsB ? 1 : LB;
    const char* src[SA + SB];
#pragma unroll
    for (int i = 0; i < SA; ++i) {
        const int at = i * kThreads + tid, r = at / OpA::kChunks;
        const int chunk = (at % OpA::kChunks) ^ OpA::swizzle(r);
        const T* a = static_cast<const T*>(p.a);
        if constexpr (kRowsA) {
            const int64_t c = min(m0 + chunk * OpA::kPerChunk, p.wa - OpA::kPerChunk);
            src[i] =
                reinterpret_cast<const char*>(a + r * p.lda + MSEL_SPAN(c, OpA::kPerChunk, p.wa));
        } else {
            const int64_t m = min(m0 + r, p.M - 1);
            src[i] = reinterpret_cast<const char*>(a + MSEL_IDX(m, p.M) * p.lda) + chunk * 16;
        }
    }
#pragma unroll
    for (int i = 0; i < SB; ++i) {
        const int at = i * kThreads + tid, r = at / OpB::kChunks;
        const int chunk = (at % OpB::kChunks) ^ OpB::swizzle(r);
        const T* b = static_cast<const T*>(p.b0);
        if constexpr (kRowsB) {
            const int64_t c = min<int64_t>(n0 + chunk * OpB::kPerChunk, p.wb - OpB::kPerChunk);
            src[SA + i] =
                reinterpret_cast<const char*>(b + r * p.ldb + MSEL_SPAN(c, OpB::kPerChunk, p.wb));
        } else {
            if (r & 32) b = static_cast<const T*>(p.b1);
            const int64_t n = min(n0 + (r >> 6) * 32 + order32(r & 31), p.N - 1);
            src[SA + i] = reinterpret_cast<const char*>(b + MSEL_IDX(n, p.N) * p.ldb) + chunk * 16;
        }
    }
    const int64_t ld_a = p.lda * static_cast<int64_t>(sizeof(T));
    const int64_t ld_b = p.ldb * static_cast<int64_t>(sizeof(T));
    const int64_t step_a = kRowsA ? kStageK<T> * ld_a : kStageBytes;
    const int64_t step_b = kRowsB ? kStageK<T> * ld_b : kStageBytes;
    const int64_t round_a = kRoundA * ld_a, round_b = kRoundB * ld_b;
    // where a stage's operands are, in bytes from the first one's, and the rows of k that its part
    // (of up to 4) has from it on
    struct Stage {
        int64_t a, b, left;
        int part;
    };
    const auto begin_part = [&](Stage& g) {
        if constexpr (KIND == Kind::kInput)  // A goes on, B is the other weight
            g.b = (g.part & 1) != 0
                      ? static_cast<const char*>(p.b1) - static_cast<const char*>(p.b0)
                      : 0;
        if constexpr (KIND == Kind::kWeights) {  // A's low parts, B again
            g.a = g.part * p.low * static_cast<int64_t>(sizeof(T));
            g.b = 0;
        }
        g.left = p.K;
    };
    // the last stage of rows of consecutive k ends with the rows: what it has in common with the
    // one before becomes 0 in LDS
    const auto end_row = [&](Stage& g) {
        if (g.left < kStageK<T>) g.a = g.b = p.K * static_cast<int64_t>(sizeof(T)) - kStageBytes;
    };
    const auto advance = [&](Stage& g) {
        g.a += step_a;
        g.b += step_b;
        g.left -= kStageK<T>;
        if constexpr (kDual) {
            end_row(g);
        } else if (g.left <= 0) {
            ++g.part;
            begin_part(g);
        }
    };
    const auto stage_at = [&](int k) {
        Stage g{k * step_a, k * step_b, p.K, 0};
        if constexpr (!kDual) {
            g.part = k / p.half;
            begin_part(g);
            k -= g.part * p.half;
            if constexpr (kRowsA) g.a += k * step_a;
            g.b += k * step_b;
        }
        g.left -= k * static_cast<int64_t>(kStageK<T>);
        if constexpr (kDual) end_row(g);
        return g;
    };
    // k that a stage has: elements of its rows (whole chunks), or rows
    const auto size_of = [&](const Stage& g) -> int {
        return g.left < kStageK<T> ? static_cast<int>(g.left) : kStageK<T>;
    };
    // kHeld: this thread's first chunk of a stage, from the stage's start, which its buffer ends
    // behind its last row: chunks of rows past the end are read as 0.  The spans of a stage are
    // below 2^32 (256 rows of 2^20 bytes).
    [[maybe_unused]] u32x4 held[kHeld ? LA + LB : 1];
    [[maybe_unused]] int from_a = 0, from_b = 0;
    if constexpr (kHeld) {
        const int ra = tid / OpA::kChunks, rb = tid / OpB::kChunks;
        const int ca = (tid % OpA::kChunks ^ OpA::swizzle(ra)) * OpA::kPerChunk;
        const int cb = (tid % OpB::kChunks ^ OpB::swizzle(rb)) * OpB::kPerChunk;
        const int64_t a0 = kRowsA ? min(m0 + ca, p.wa - OpA::kPerChunk) : ca;
        const int64_t b0 = min<int64_t>(n0 + cb, p.wb - OpB::kPerChunk);
        from_a = static_cast<int>((ra * p.lda + a0) * sizeof(T));
        from_b = static_cast<int>((rb * p.ldb + b0) * sizeof(T));
    }
    const auto buffer_of = [](const void* base, int64_t bytes) {
        const uint32_t n = bytes < 0xffffffff ? static_cast<uint32_t>(bytes) : 0xffffffffu;
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(n),
                                                 0x00020000);
    };
    // loads [i0, i1) of a stage
    const auto load_part = [&](const Stage& stage, int buf, int i0, int i1) {
        if constexpr (kHeld) {
            const char* const a =
                static_cast<const char*>(p.a) + stage.a + (kRowsA ? 0 : m0 * ld_a);
            const char* const b = static_cast<const char*>(p.b0) + stage.b;
            const auto from_of_a =
                buffer_of(a, kRowsA ? stage.left * ld_a : (p.M - m0) * ld_a - stage.a);
            const auto from_of_b = buffer_of(b, stage.left * ld_b);
            const int to_a = static_cast<int>(round_a), to_b = static_cast<int>(round_b);
#pragma unroll
            for (int i = i0; i < i1; ++i)
                held[i] = __builtin_bit_cast(
                    u32x4, i < LA ? __builtin_amdgcn_raw_buffer_load_b128(
                                        from_of_a, from_a + i * to_a, 0, 0)
                                  : __builtin_amdgcn_raw_buffer_load_b128(
                                        from_of_b, from_b + (i - LA) * to_b, 0, 0));
        } else {
            const int size = size_of(stage);
            // rows of this thread's first chunks behind the stage's end
            [[maybe_unused]] const int past_a = tid / OpA::kChunks - size;
            [[maybe_unused]] const int past_b = tid / OpB::kChunks - size;
#pragma unroll
            for (int i = 0; i < LA + LB; ++i) {
                if (i < i0 || i >= i1) continue;
                const bool a = i < LA;
                const char* g = a ? src[kRowsA ? 0 : i] + (stage.a + (kRowsA ? i * round_a : 0))
                                  : src[SA + (kRowsB ? 0 : i - LA)] +
                                        (stage.b + (kRowsB ? (i - LA) * round_b : 0));
                if ((a ? kRowsA : kRowsB) && size < kStageK<T>) {  // uniform
                    const int past = a ? past_a + i * kRoundA : past_b + (i - LA) * kRoundB;
                    if (past >= 0) g -= (past + 1) * (a ? ld_a : ld_b);
                }
                const int at = buf * kStage + (i * kThreads + wave * 64) * 16;
                __builtin_amdgcn_global_load_lds((GlobalVoid*)g, (LdsVoid*)(lds + at), 16, 0, 0);
            }
        }
    };
    // kHeld: loads [i0, i1) go to LDS
    const auto write_part = [&](int buf, int i0, int i1) {
#pragma unroll
        for (int i = i0; i < i1; ++i)
            *reinterpret_cast<u32x4*>(lds + buf * kStage + (i * kThreads + tid) * 16) = held[i];
    };

    f32x16 acc[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    // fp32: the sums of the stages before the last kPartStages (the largest tiles have no more)
    constexpr bool kParts = sizeof(T) == 4 && MI < 4;
    f32x16 sum[kParts ? MI : 1][2];
    const auto add_part = [&](bool first_one) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    sum[i][j][e] = first_one ? acc[i][j][e] : sum[i][j][e] + acc[i][j][e];
                    acc[i][j][e] = 0.0f;
                }
    };

    // kGateGrad: dout's tile in the order in which the results go out; loaded before the product
    // where the registers for it are there (32 in bf16)
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    constexpr int kOut = BM * CW / VE / kThreads;
    RawVec<T, VE> dout[KIND == Kind::kGateGrad ? kOut : 1];
    const auto load_dout = [&] {
#pragma unroll
        for (int i = 0; i < kOut; ++i) {
            const int at = i * kThreads + tid, n = n0 + at % (CW / VE) * VE;
            const int64_t m = min(m0 + at / (CW / VE), p.M - 1);
            const T* row = static_cast<const T*>(p.dout) + MSEL_IDX(m, p.M) * p.N;
            if (n + VE <= p.N)
                dout[i] = ld_raw<T, VE>(row + MSEL_SPAN(n, VE, p.N));
            else
                dout[i] = ld_part<T, VE>(row + n, p.N - n);
        }
    };
    if constexpr (KIND == Kind::kGateGrad && sizeof(T) == 2)
        if (p.part == nullptr) load_dout();

    const int first = split * p.per_split, last = min(p.stages, first + p.per_split);
    // waits for stage k, which has `after` loads behind it; what it has too much becomes 0
    const auto enter_stage = [&](int k, int size, auto after) {
        if constexpr (kHeld) {
            barrier_of_lds();
            return;
        }
        barrier_after<decltype(after)::value>();
        if (size == kStageK<T>) return;  // uniform
        const u32x4 zero = {0, 0, 0, 0};
        char* at = lds + ((k - first) & 1) * kStage;
        if constexpr (kDual) {  // rows of both operands alike
            for (int i = tid; i < kStage / 16; i += kThreads)
                if ((i % 8 ^ OpA::swizzle(i / 8)) < 8 - size / OpA::kPerChunk)
                    *reinterpret_cast<u32x4*>(at + i * 16) = zero;
        } else {
            if (kRowsA)
                for (int i = size * OpA::kChunks + tid; i < OpA::kBytes / 16; i += kThreads)
                    *reinterpret_cast<u32x4*>(at + i * 16) = zero;
            for (int i = size * OpB::kChunks + tid; i < OpB::kBytes / 16; i += kThreads)
                *reinterpret_cast<u32x4*>(at + OpA::kBytes + i * 16) = zero;
        }
        __syncthreads();
    };
    u32x4 fa[2][MI], fb[2][2];  // fragments of a step and of the next
    const auto read_step = [&](int k, int s, int to) {
        const char* sa = lds + ((k - first) & 1) * kStage;
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[to][i] = OpA::read(sa, wm * MI + i, s, lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) fb[to][j] = OpB::read(sa + OpA::kBytes, wn * 2 + j, s, lane);
    };
    Stage loading = stage_at(first);  // the last stage whose loads are out
    const int first_size = size_of(loading);
    load_part(loading, 0, 0, LA + LB);
    if constexpr (kHeld) {
        write_part(0, 0, LA + LB);
        if (first + 1 < last) advance(loading);
        load_part(loading, 1, 0, LA + LB);
        enter_stage(first, first_size, std::integral_constant<int, 0>());
    } else if (first + 1 < last) {
        advance(loading);
        load_part(loading, 1, 0, LA + LB);
        enter_stage(first, first_size, std::integral_constant<int, LA + LB>());
    } else {
        enter_stage(first, first_size, std::integral_constant<int, 0>());
    }
    read_step(first, 0, 0);
    // A stage's loads go out between the MFMAs, half of them in the step before it is entered and
    // half in the one after: all at once they would hold up the wavefronts that issue them.
    constexpr int kHalf = (LA + LB) / 2, kPer = kHalf / MI;
    static_assert(kPer * MI * 2 == LA + LB, "whole parts");
    for (int k = first; k < last; ++k) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int cur = s & 1;
            const auto mfmas = [&](int i, int j) {
                mfma_step(static_cast<const T*>(nullptr), fb[cur][j], fa[cur][i], acc[i][j]);
            };
            // the first MFMA waits for fragments that were read during the step before; the next
            // reads go out behind it, or it would wait for them too (777 x 1000 -> 2603 in fp32,
            // backward: 288 us so, 280 this way)
            mfmas(0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (s + 1 < kSteps) {
                read_step(k, s + 1, cur ^ 1);
            } else if (kHeld || k + 1 < last) {
                enter_stage(k + 1, size_of(loading), std::integral_constant<int, 0>());
                read_step(k + 1, 0, cur ^ 1);
            }
            if (!kHeld && s + 1 == kSteps && k + 2 < last) advance(loading);
            if (kHeld && s == 0 && k + 2 < last) advance(loading);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
#pragma unroll
                for (int j = i == 0 ? 1 : 0; j < 2; ++j) mfmas(i, j);
                if constexpr (kHeld) {
                    // stage k + 1 goes to LDS and k + 2 is loaded behind it, half of both in steps
                    // 0 and 1 (past the last stage that one again, to no use)
                    if (s < 2) {
                        const int i0 = s * kHalf + i * kPer;
                        write_part((k + 1 - first) & 1, i0, i0 + kPer);
                        load_part(loading, 0, i0, i0 + kPer);
                    }
                } else {
                    if (s + 1 == kSteps && k + 2 < last)
                        load_part(loading, (k - first) & 1, i * kPer, (i + 1) * kPer);
                    if (s == 0 && k > first && k + 1 < last)
                        load_part(loading, (k + 1 - first) & 1, kHalf + i * kPer,
                                  kHalf + (i + 1) * kPer);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (kParts)
            if ((k - first) % kPartStages == kPartStages - 1) add_part(k - first < kPartStages);
    }
    if constexpr (kParts) {
        if (last - first >= kPartStages) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] += sum[i][j];
        }
    }
    __syncthreads();  // the ring becomes the tile on its way out

    // lane l holds 16 columns from 16 (l / 32) on of row l % 32 of its fragments
    const int h16 = (lane >> 5) * 16, r0 = wm * MI * 32 + (lane & 31);
    const auto values = [](const f32x16& a, float (&v)[16]) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = a[e];
    };
    // rows of a tile of W columns of type U to dst(row of C, first column in the tile, chunk)
    const auto send = [&](auto tile, auto dst) {
        using Tile = decltype(tile);
        __syncthreads();
        for (int at = tid; at < BM * Tile::kChunks; at += kThreads) {
            const int r = at / Tile::kChunks, c = at % Tile::kChunks;
            if (m0 + r < p.M) dst(m0 + r, c * Tile::kPerChunk, lds + Tile::place(r, c));
        }
    };
    if constexpr (kDual) {
        using Tile = OutTile<T, CW>;
        static_assert(BM * CW * sizeof(T) <= kRing * kStage, "the tile fits where the ring was");
        const int col = wn * 32 + h16;
        const auto to = [&](int shift, int cols) {
            return [&, shift, cols](int64_t m, int c, const char* from) {
                RawVec<T, VE> raw;
                __builtin_memcpy(&raw, from, 16);
                store_columns<T, VE>(static_cast<T*>(p.c0) + m * p.ldc + shift, n0 + c, cols, raw);
            };
        };
        if (p.part != nullptr) {
            using Part = OutTile<float, CW>;
            static_assert(BM * CW * sizeof(float) <= kRing * kStage, "fits");
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (j > 0) __syncthreads();
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    float v[16];
                    values(acc[i][j], v);
                    Part::put(lds, r0 + i * 32, col, v);
                }
                send(Part(), [&](int64_t m, int c, const char* from) {
                    RawVec<float, 4> raw;
                    __builtin_memcpy(&raw, from, 16);
                    float* row = p.part + ((split * 2 + j) * p.M + m) * p.N;
                    store_columns<float, 4>(row, n0 + c, p.N, raw);
                });
            }
        } else if constexpr (KIND == Kind::kGate) {
            with_act(p.gelu, [&](auto gelu) {
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    float g[16], u[16];
                    values(acc[i][0], g);
                    values(acc[i][1], u);
#pragma unroll
                    for (int e = 0; e < 16; ++e) g[e] = act_of<gelu.value>(g[e]) * u[e];
                    Tile::put(lds, r0 + i * 32, col, g);
                }
            });
            send(Tile(), to(0, p.N));
        } else {
            if constexpr (sizeof(T) == 4) load_dout();
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
                const int at = i * kThreads + tid;
                __builtin_memcpy(lds + Tile::place(at / Tile::kChunks, at % Tile::kChunks),
                                 &dout[i], 16);
            }
            __syncthreads();
            // dG over dout, a lane's own columns; dU waits where U was (and dG where G was, for its
            // low part: the largest tiles have no registers for that)
            constexpr bool kLow = sizeof(T) == 2 && MI < 4;
            with_act(p.gelu, [&](auto gelu) {
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    float d[16], g[16], u[16];
                    Tile::get(lds, r0 + i * 32, col, d);
                    values(acc[i][0], g);
                    values(acc[i][1], u);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float v, slope;
                        act_grad<gelu.value>(g[e], v, slope);
                        g[e] = d[e] * u[e] * slope;
                        u[e] = d[e] * v;
                    }
                    // columns behind the weights' last row are 0: the next products read them
                    if (n0 + CW > p.N) {  // uniform
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const bool in = n0 + col + e < p.N;
                            g[e] = in ? g[e] : 0.0f;
                            u[e] = in ? u[e] : 0.0f;
                        }
                    }
                    Tile::put(lds, r0 + i * 32, col, g);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        if constexpr (kLow) acc[i][0][e] = g[e];
                        acc[i][1][e] = u[e];
                    }
                }
            });
            send(Tile(), to(0, p.hp));
            const auto put_all = [&](auto j, auto value) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    float v[16];
                    values(acc[i][j.value], v);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = value(v[e]);
                    Tile::put(lds, r0 + i * 32, col, v);
                }
            };
            const std::integral_constant<int, 0> dg;
            const std::integral_constant<int, 1> du;
            put_all(du, [](float v) { return v; });
            send(Tile(), to(p.hp, p.hp));
            if constexpr (kLow) {
                if (p.with_low) {  // uniform
                    put_all(dg, [](float v) { return rest_of(v); });
                    send(Tile(), to(2 * p.hp, p.hp));
                    put_all(du, [](float v) { return rest_of(v); });
                    send(Tile(), to(3 * p.hp, p.hp));
                }
            }
        }
    } else {
        // fp32 in two halves: the first 32 of each wavefront's 64 columns, then the others
        const auto halves = [&](auto row_of) {
            using Tile = OutTile<float, BN / 2>;
            static_assert(BM * BN / 2 * sizeof(float) <= kRing * kStage, "fits");
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (j > 0) __syncthreads();
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    float v[16];
                    values(acc[i][j], v);
                    Tile::put(lds, r0 + i * 32, wn * 32 + h16, v);
                }
                send(Tile(), [&](int64_t m, int c, const char* from) {
                    float* row = row_of(m);
                    RawVec<float, 4> raw;
                    __builtin_memcpy(&raw, from, 16);
                    const int n = n0 + (c >> 5) * 64 + j * 32 + (c & 31);
                    if (row != nullptr) store_columns<float, 4>(row, n, p.N, raw);
                });
            }
        };
        const auto row_of = [&](int64_t m) -> T* {
            return m < p.rows0    ? static_cast<T*>(p.c0) + m * p.ldc
                   : m >= p.split ? static_cast<T*>(p.c1) + (m - p.split) * p.ldc
                                  : nullptr;
        };
        if (p.part != nullptr) {
            halves([&](int64_t m) { return p.part + (split * p.M + m) * p.N; });
        } else if constexpr (sizeof(T) == 4) {
            halves(row_of);
        } else {
            using Tile = OutTile<T, BN>;
            static_assert(BM * BN * sizeof(T) <= kRing * kStage, "fits");
#pragma unroll
            for (int i = 0; i < MI; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[16];
                    values(acc[i][j], v);
                    Tile::put(lds, r0 + i * 32, wn * 64 + j * 32 + h16, v);
                }
            }
            send(Tile(), [&](int64_t m, int c, const char* from) {
                T* row = row_of(m);
                RawVec<T, VE> raw;
                __builtin_memcpy(&raw, from, 16);
                if (row != nullptr) store_columns<T, VE>(row, n0 + c, p.N, raw);
            });
        }
    }
}

// Few tokens: a block for 8 columns of both weights, whose 16 rows go from memory into the MFMA's
// registers, each read once for up to 16 NT tokens; its wavefronts take the chunks of k in turn and
// their sums are added in LDS.  HBM bounds it: 8 tokens of 2048 -> 5632 read 46 MB.  (16 columns a
// block, the weights in MFMAs of their own: 352 blocks for 256 CUs there, 12.9 us.)
template <typename T, int NT>
__global__ __launch_bounds__(256) void skinny_kernel(ProductParams p) {
    constexpr int kWaves = 4, kCols = 8;
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    constexpr int kChunk = 8 * VE;  // of k per wavefront: two vectors a lane, 128 bytes of a row
    constexpr int kAhead = 4;       // chunks on their way together
    typedef float f32x4_t __attribute__((ext_vector_type(4)));
    __shared__ float sums[kWaves][NT][16][16];
    const int lane = lane_id(), wave = threadIdx.x >> 6;
    const int n0 = static_cast<int>(xcd_order(blockIdx.x, gridDim.x)) * kCols;
    const int K = static_cast<int>(p.K);
    // rows 0..7 of the MFMA are Wg's, 8..15 Wu's; rows past the end repeat the last one, and their
    // results are not stored
    const int64_t n = MSEL_IDX(min(n0 + (lane & 7), p.N - 1), p.N);
    const T* const w = static_cast<const T*>((lane & 8) ? p.b1 : p.b0) + n * p.ldb;
    const T* x[NT];
    f32x4_t acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t m = MSEL_IDX(min<int64_t>(t * 16 + (lane & 15), p.M - 1), p.M);
        x[t] = static_cast<const T*>(p.a) + m * p.lda;
        acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const auto load = [&](const T* row, int k) {  // columns past the end are 0
        if (k + VE <= K) return ld_raw<T, VE>(row + MSEL_SPAN(k, VE, K));
        return ld_part<T, VE>(row + k, K - k);
    };
    const auto product = [&](const RawVec<T, VE>& a, const RawVec<T, VE>& b, f32x4_t& c) {
        if constexpr (sizeof(T) == 2) {
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, a.w), __builtin_bit_cast(bf16x8, b.w), c, 0, 0, 0);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w[e]),
                                                         __uint_as_float(b.w[e]), c, 0, 0, 0);
        }
    };
    // lane l: row l % 16, 2 vectors from 2 VE (l / 16) on of a chunk
    const int at = (lane >> 4) * 2 * VE;
    for (int k0 = wave * kChunk; k0 < K; k0 += kAhead * kWaves * kChunk) {
        RawVec<T, VE> vw[kAhead][2], vx[kAhead][2][NT];
#pragma unroll
        for (int c = 0; c < kAhead; ++c) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int k = k0 + c * kWaves * kChunk + at + v * VE;
                vw[c][v] = load(w, k);
#pragma unroll
                for (int t = 0; t < NT; ++t) vx[c][v][t] = load(x[t], k);
            }
        }
#pragma unroll
        for (int c = 0; c < kAhead; ++c)
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int t = 0; t < NT; ++t) product(vw[c][v], vx[c][v][t], acc[t]);
    }
    // lane l holds token l % 16 and rows 4 (l / 16) + 0..3
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[wave][t][4 * (lane >> 4) + e][lane & 15] = acc[t][e];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 16 * kCols; i += 256) {
        const int m = i / kCols, c = i % kCols;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            g += sums[v][m >> 4][c][m & 15];
            u += sums[v][m >> 4][8 + c][m & 15];
        }
        if (m < p.M && n0 + c < p.N) {
            T* row = static_cast<T*>(p.c0) + m * p.ldc;
            with_act(p.gelu, [&](auto gelu) {
                Elem<T>::store1(row + MSEL_IDX(n0 + c, p.N), act_of<gelu.value>(g) * u);
            });
        }
    }
}

// Rows [0, rows0) of C to c0 and those from `split` on to c1, as sums of their parts in order.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(const float* part, int splits, int64_t M, int N,
                                                   int64_t rows0, int64_t split, T* c0, T* c1) {
    const int64_t n = M * N, end0 = rows0 * N, n1 = (M - split) * N;
    const int64_t first = blockIdx.y == 0 ? 0 : split * N, len = blockIdx.y == 0 ? end0 : n1;
    T* const c = blockIdx.y == 0 ? c0 : c1;
    const float* const from = part + first;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < len;
         i += static_cast<int64_t>(gridDim.x) * 1024) {
        if (i + 4 <= len) {
            float v[4] = {};
            for (int s = 0; s < splits; ++s) {
                float w[4];
                to_f32<float, 4>(
                    ld_raw<float, 4>(from + s * n + MSEL_SPAN(i, 4, n - first)), w);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += w[e];
            }
            if constexpr (sizeof(T) == 4) {
                st_vec<T, 4>(c + MSEL_SPAN(i, 4, len), v);
            } else {
                const uint32_t w[2] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                __builtin_memcpy(c + MSEL_SPAN(i, 4, len), w, 8);
            }
        } else {
            for (int e = 0; i + e < len; ++e) {
                float v = 0.0f;
                for (int s = 0; s < splits; ++s) v += from[s * n + MSEL_IDX(i + e, n - first)];
                Elem<T>::store1(c + MSEL_IDX(i + e, len), v);
            }
        }
    }
}

// What comes of G and U whose stages were split: sums of their parts in order, then as in the
// product's own epilogue.  Four columns a thread.
template <typename T, Kind KIND>
__global__ __launch_bounds__(256) void gate_join_kernel(ProductParams p) {
    constexpr bool kGrad = KIND == Kind::kGateGrad;
    const int cols = kGrad ? p.hp : p.N, per = (cols + 3) / 4;
    const int64_t n = p.M * per;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t m = MSEL_IDX(i / per, p.M);
        const int c = static_cast<int>(i - m * per) * 4, valid = p.N - c;  // beyond N all is 0
        float sums[2][4] = {};
        for (int s = 0; s < p.splits; ++s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float* const from = p.part + ((s * 2 + j) * p.M + m) * p.N + c;
                float v[4];
                to_f32<float, 4>(ld_part<float, 4>(from, valid), v);
#pragma unroll
                for (int e = 0; e < 4; ++e) sums[j][e] += v[e];
            }
        }
        T* const out = static_cast<T*>(p.c0) + m * p.ldc + c;
        const auto put = [&](int shift, const float (&v)[4]) {
            const RawVec<T, 4> raw = from_f32<T, 4>(v);
            if constexpr (kGrad)
                st_raw<T, 4>(out + shift, raw);
            else
                st_part<T, 4>(out, raw, valid);
        };
        with_act(p.gelu, [&](auto gelu) {
            if constexpr (!kGrad) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = act_of<gelu.value>(sums[0][e]) * sums[1][e];
                put(0, v);
            } else {
                float d[4], g[4], u[4];
                to_f32<T, 4>(ld_part<T, 4>(static_cast<const T*>(p.dout) + m * p.N + c, valid), d);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v, slope;
                    act_grad<gelu.value>(sums[0][e], v, slope);
                    g[e] = d[e] * sums[1][e] * slope;
                    u[e] = d[e] * v;
                }
                put(0, g);
                put(p.hp, u);
                if constexpr (sizeof(T) == 2) {
                    if (p.with_low) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            g[e] = rest_of(g[e]);
                            u[e] = rest_of(u[e]);
                        }
                        put(2 * p.hp, g);
                        put(3 * p.hp, u);
                    }
                }
            }
        });
    }
}

// The operands' rows, padded with zeros to whole chunks of 16 bytes: dst[r][c] = src[r][c] for c <
// cols, 0 up to ldd; one operand per blockIdx.y.
struct PadParams {
    const void* src[3];
    void* dst[3];
    int64_t rows[3];
    int cols, ldd;
};
template <typename T>
__global__ __launch_bounds__(256) void pad_kernel(PadParams p) {
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    const T* const src = static_cast<const T*>(p.src[blockIdx.y]);
    T* const dst = static_cast<T*>(p.dst[blockIdx.y]);
    const int per = p.ldd / VE;
    const int64_t n = p.rows[blockIdx.y] * per;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = i / per;
        const int c = static_cast<int>(i - r * per) * VE;
        const T* row = src + MSEL_IDX(r, p.rows[blockIdx.y]) * p.cols;
        const RawVec<T, VE> v = c + VE <= p.cols ? ld_raw<T, VE>(row + MSEL_SPAN(c, VE, p.cols))
                                                 : ld_part<T, VE>(row + c, p.cols - c);
        st_raw<T, VE>(dst + MSEL_IDX(i, n) * VE, v);
    }
}

constexpr unsigned kMaxBlocks = 1u << 20;

// ---- plans -------------------------------------------------------------------------------------

int64_t over(int64_t n, int64_t q) { return (n + q - 1) / q; }

// Tiles of a product and how its stages are split over blocks.
struct ProductPlan {
    int tile;    // 0: 256 x 256, 1: 128 x 128, 2: 64 x 128
    int splits;
};

// The cheapest by a model in cycles: the blocks of a CU take turns on its matrix cores, at the
// share of the peak that such tiles reach (below, fitted to measured products), but a stage takes
// no less than the way of its loads, which the blocks that a CU holds share; then a fixed part per
// block, and for split stages the join's launch (a call's second one in the forward) and the parts'
// way through the last-level cache.  dG and dU of 16384 x 768 -> 2048: 256 x 256 158 us, 128 x 128
// 185.  Backward of 1024 x 768 -> 2048: dx alone 38 us, its sums not split 49; forward of 181 x
// 2880 -> 64 in fp32: 19 us, not split 103.
ProductPlan plan_product(Kind kind, int64_t M, int64_t cols, int stages, bool bf16,
                         int first_tile = 0) {
    constexpr int rows_of[] = {256, 128, 64}, cols_of[] = {256, 128, 128}, held[] = {1, 2, 3};
    constexpr double share16[] = {0.8, 0.52, 0.5}, share32[] = {0.74, 0.74, 0.7};
    constexpr int kCus = 256;
    constexpr double kLoads = 2000.0;
    ProductPlan best{1, 1};
    double least = 0.0;
    for (int t = first_tile; t < 3; ++t) {
        const int64_t tiles = over(M, rows_of[t]) * over(cols, cols_of[t]);
        const double area = rows_of[t] * cols_of[t];
        const double stage = area * (bf16 ? 64 / 2048.0 / share16[t] : 32 / 128.0 / share32[t]);
        for (int s = 1; s <= 16 && (s == 1 || stages / s >= 4); ++s) {
            if (!bf16 && t == 0 && over(stages, s) > kPartStages) continue;
            const int64_t turns = over(tiles * s, kCus), full = turns / held[t];
            const int rest = static_cast<int>(turns % held[t]);
            const double a_stage = full * std::max(held[t] * stage, kLoads) +
                                   (rest > 0 ? std::max(rest * stage, kLoads) : 0.0);
            double cost = over(stages, s) * a_stage + turns * (1000.0 + area / 12.0);
            if (s > 1)
                cost += (dual(kind) ? 18000.0 : 12000.0) +
                        static_cast<double>(s) * M * cols * 8 / 6000.0;
            if (least == 0.0 || cost < least) {
                least = cost;
                best = {t, s};
            }
        }
    }
    best.splits = static_cast<int>(over(stages, over(stages, best.splits)));
    return best;
}

template <typename T, int WM, int WN, int MI, Kind KIND>
hipError_t launch_tiles(ProductParams p, int splits, hipStream_t stream) {
    constexpr int BM = WM * MI * 32, BN = WN * 64;
    constexpr int bytes = kRing * (BM + BN) * kStageBytes;
    const int bn = dual(KIND) ? BN / 2 : BN;
    p.tm = static_cast<int>(over(p.M, BM));
    p.tn = static_cast<int>(over(KIND == Kind::kGateGrad ? p.hp : p.N, bn));
    p.splits = splits;
    p.per_split = static_cast<int>(over(p.stages, splits));
    const hipError_t e = allow_dynamic_lds<product_kernel<T, WM, WN, MI, KIND>>(bytes);
    if (e != hipSuccess) return e;
    const int64_t blocks = static_cast<int64_t>(p.tm) * p.tn * splits;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(blocks, kMaxBlocks)),
                    static_cast<unsigned>(over(blocks, kMaxBlocks)));
    hipLaunchKernelGGL((product_kernel<T, WM, WN, MI, KIND>), grid, dim3(WM * WN * 64), bytes,
                       stream, p);
    return hipGetLastError();
}

template <typename T, Kind KIND>
hipError_t launch_product(const ProductParams& p, const ProductPlan& q, hipStream_t stream) {
    switch (q.tile) {
        case 0: return launch_tiles<T, 2, 4, 4, KIND>(p, q.splits, stream);
        case 1: return launch_tiles<T, 2, 2, 2, KIND>(p, q.splits, stream);
        default: return launch_tiles<T, 2, 2, 1, KIND>(p, q.splits, stream);
    }
}

// Those of G and U: their parts in `part`, then what comes of their sums.
template <typename T, Kind KIND>
hipError_t launch_gate(ProductParams p, const ProductPlan& q, float* part, hipStream_t stream) {
    if (q.splits == 1) return launch_product<T, KIND>(p, q, stream);
    p.part = part;
    p.splits = q.splits;
    const hipError_t e = launch_product<T, KIND>(p, q, stream);
    if (e != hipSuccess) return e;
    const int64_t units = p.M * over(KIND == Kind::kGateGrad ? p.hp : p.N, 4);
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(over(units, 256), kMaxBlocks)));
    hipLaunchKernelGGL((gate_join_kernel<T, KIND>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

// A product whose stages may be split: its parts in `part`, then their sum.
template <typename T, Kind KIND>
hipError_t launch_split(ProductParams p, const ProductPlan& q, float* part, hipStream_t stream) {
    if (q.splits == 1) return launch_product<T, KIND>(p, q, stream);
    p.part = part;
    const hipError_t e = launch_product<T, KIND>(p, q, stream);
    if (e != hipSuccess) return e;
    const int64_t blocks = std::min<int64_t>(over(p.rows0 * p.N, 1024), kMaxBlocks);
    hipLaunchKernelGGL(join_kernel<T>, dim3(static_cast<unsigned>(blocks), p.split < p.M ? 2 : 1),
                       dim3(256), 0, stream, part, q.splits, p.M, p.N, p.rows0, p.split,
                       static_cast<T*>(p.c0), static_cast<T*>(p.c1));
    return hipGetLastError();
}

// Up to so many tokens times the smaller width dG and dU are held in two bf16 numbers each, the
// value rounded and what that left, beyond it in one, as the operands of the next products.  One
// number leaves results off by 2.33e-3 of their norm at every size, two by 1.66e-3, which is the
// rounding of the results themselves.  The second one doubles dx's and the weights' products: 4 x
// 768 -> 2048 29 us, 26 with one, 8 x 2048 -> 5632 59, 50, 16384 x 768 -> 2048 593, 342.  So it is
// there where launches are most of the call.
constexpr int64_t kFew = 4096;

// Parts of the workspace: offsets in bytes, absent parts take none.
struct MlpSpace {
    // rows of the operands (whole chunks, at least a stage), the hidden width in stages
    int64_t dp, hp;
    size_t x = 0, wg = 0, wu = 0, dgu = 0, part = 0, all = 0;
    int parts_of = 1;  // bf16 numbers that dG and dU are held in, each
    ProductPlan gate, input, weights;
    MlpSpace(const MlpParams& p, bool bf16, bool bwd) {
        const size_t elem = bf16 ? 2 : 4;
        const int64_t q = kStageBytes / static_cast<int64_t>(elem);
        const int64_t chunk = 16 / static_cast<int64_t>(elem);
        dp = p.D < q ? q : over(p.D, chunk) * chunk;
        hp = over(p.F, q) * q;
        const auto take = [&](size_t bytes) {
            const size_t at = all;
            all += (bytes + 255) / 256 * 256;
            return at;
        };
        if (dp != p.D) {
            x = take(static_cast<size_t>(p.M * dp) * elem);
            wg = take(static_cast<size_t>(p.F * dp) * elem);
            wu = take(static_cast<size_t>(p.F * dp) * elem);
        }
        if (bwd && bf16 && p.M * std::min(p.D, p.F) <= kFew) parts_of = 2;
        gate = plan_product(bwd ? Kind::kGateGrad : Kind::kGate, p.M, 2 * (bwd ? hp : p.F),
                            static_cast<int>(over(dp, q)), bf16, parts_of > 1 ? 1 : 0);
        size_t parts = 0;  // of one product at a time
        if (gate.splits > 1) parts = static_cast<size_t>(gate.splits) * 2 * p.M * p.F;
        if (!bwd) {
            part = take(parts * sizeof(float));
            return;
        }
        dgu = take(static_cast<size_t>(p.M * 2 * parts_of * hp) * elem);
        input = plan_product(Kind::kInput, p.M, p.D, static_cast<int>(2 * parts_of * hp / q), bf16);
        weights = plan_product(Kind::kWeights, hp + p.F, p.D,
                               static_cast<int>(parts_of * over(p.M, q)), bf16);
        if (input.splits > 1)
            parts = std::max(parts, static_cast<size_t>(input.splits) * p.M * p.D);
        if (weights.splits > 1)
            parts = std::max(parts, static_cast<size_t>(weights.splits) * (hp + p.F) * p.D);
        part = take(parts * sizeof(float));
    }
};

// The operands with rows of whole chunks, at least a stage.
struct Padded {
    const void* x;
    const void* wg;
    const void* wu;
};
template <typename T>
Padded padded(const MlpParams& p, const MlpSpace& w, hipStream_t stream) {
    if (w.dp == p.D) return {p.x, p.wg, p.wu};
    char* const ws = static_cast<char*>(p.ws);
    const PadParams q{{p.x, p.wg, p.wu}, {ws + w.x, ws + w.wg, ws + w.wu}, {p.M, p.F, p.F}, p.D,
                      static_cast<int>(w.dp)};
    const int64_t blocks = over(std::max<int64_t>(p.M, p.F) * w.dp * sizeof(T), 256 * 16);
    hipLaunchKernelGGL(pad_kernel<T>,
                       dim3(static_cast<unsigned>(std::min<int64_t>(blocks, kMaxBlocks)), 3),
                       dim3(256), 0, stream, q);
    return {ws + w.x, ws + w.wg, ws + w.wu};
}

template <typename T>
ProductParams gate_params(const MlpParams& p, const MlpSpace& w, const Padded& o) {
    ProductParams q{};
    q.M = p.M;
    q.N = p.F;
    q.K = w.dp;
    q.stages = q.half = static_cast<int>(over(w.dp, kStageK<T>));
    q.lda = q.ldb = w.dp;
    q.a = o.x;
    q.b0 = o.wg;
    q.b1 = o.wu;
    q.gelu = p.gelu;
    return q;
}

// Whether the skinny kernel takes a call: up to 16 tokens, and up to 32 (48 in fp32) where the
// weights are small, where the launch of the parts' join would show (768 -> 2048 in bf16: 10 us for
// 32 tokens, the tiles 14; 2048 -> 5632: 11.5 for 8, 13 for 16, 19 for 32, the tiles 15.5, 16 and
// 17; 4096 -> 8192: 30 for 16, 44 for 32, the tiles 27 and 28).
bool is_skinny(const MlpParams& p, bool bf16) {
    const int64_t weights = int64_t(2) * p.D * p.F * (bf16 ? 2 : 4);
    return p.M <= 16 || (p.M <= (bf16 ? 32 : 48) && weights <= int64_t(32) << 20);
}

template <typename T>
hipError_t forward_skinny(const MlpParams& p, hipStream_t stream) {
    ProductParams q{};
    q.M = p.M;
    q.N = p.F;
    q.K = q.lda = q.ldb = p.D;
    q.a = p.x;
    q.b0 = p.wg;
    q.b1 = p.wu;
    q.c0 = p.out;
    q.ldc = p.F;
    q.gelu = p.gelu;
    const dim3 grid(static_cast<unsigned>(over(p.F, 8))), block(256);
    switch (over(p.M, 16)) {
        case 1: hipLaunchKernelGGL((skinny_kernel<T, 1>), grid, block, 0, stream, q); break;
        case 2: hipLaunchKernelGGL((skinny_kernel<T, 2>), grid, block, 0, stream, q); break;
        default:
            if constexpr (sizeof(T) == 4)
                hipLaunchKernelGGL((skinny_kernel<T, 3>), grid, block, 0, stream, q);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t forward(const MlpParams& p, hipStream_t stream) {
    if (is_skinny(p, sizeof(T) == 2)) return forward_skinny<T>(p, stream);
    const MlpSpace w(p, sizeof(T) == 2, false);
    ProductParams q = gate_params<T>(p, w, padded<T>(p, w, stream));
    q.c0 = p.out;
    q.ldc = p.F;
    return launch_gate<T, Kind::kGate>(
        q, w.gate, reinterpret_cast<float*>(static_cast<char*>(p.ws) + w.part), stream);
}

template <typename T>
hipError_t backward(const MlpParams& p, hipStream_t stream) {
    const MlpSpace w(p, sizeof(T) == 2, true);
    char* const ws = static_cast<char*>(p.ws);
    float* const part = reinterpret_cast<float*>(ws + w.part);
    const Padded o = padded<T>(p, w, stream);
    ProductParams q = gate_params<T>(p, w, o);
    q.c0 = ws + w.dgu;
    q.ldc = 2 * w.parts_of * w.hp;
    q.hp = static_cast<int>(w.hp);
    q.with_low = w.parts_of > 1;
    q.dout = p.dout;
    hipError_t e = launch_gate<T, Kind::kGateGrad>(q, w.gate, part, stream);
    if (e != hipSuccess) return e;
    if (p.dx != nullptr) {
        ProductParams r{};
        r.M = r.rows0 = r.split = p.M;
        r.N = p.D;
        r.K = p.F;
        r.half = static_cast<int>(w.hp / kStageK<T>);
        r.stages = 2 * w.parts_of * r.half;
        r.a = ws + w.dgu;
        r.lda = 2 * w.parts_of * w.hp;
        r.b0 = o.wg;
        r.b1 = o.wu;
        r.ldb = r.wb = w.dp;
        r.c0 = p.dx;
        r.ldc = p.D;
        e = launch_split<T, Kind::kInput>(r, w.input, part, stream);
        if (e != hipSuccess) return e;
    }
    if (p.dwg != nullptr) {
        ProductParams r{};
        r.M = w.hp + p.F;  // dG's columns, a gap up to hp, dU's
        r.rows0 = p.F;
        r.split = w.hp;
        r.N = p.D;
        r.K = p.M;
        r.half = static_cast<int>(over(p.M, kStageK<T>));
        r.stages = w.parts_of * r.half;
        r.a = ws + w.dgu;
        r.wa = r.low = 2 * w.hp;
        r.lda = 2 * w.parts_of * w.hp;
        r.b0 = r.b1 = o.x;
        r.ldb = r.wb = w.dp;
        r.ldc = p.D;
        r.c0 = p.dwg;
        r.c1 = p.dwu;
        e = launch_split<T, Kind::kWeights>(r, w.weights, part, stream);
    }
    return e;
}

}  // namespace

size_t mlp_fwd_workspace_bytes(const MlpParams& p, bool bf16) {
    if (is_skinny(p, bf16)) return 0;
    return MlpSpace(p, bf16, false).all;
}

size_t mlp_bwd_workspace_bytes(const MlpParams& p, bool bf16) {
    return MlpSpace(p, bf16, true).all;
}

void mlp_tiles(int64_t tokens, int dim, int hidden, bool bf16, int* tiles) {
    MlpParams p{};
    p.M = tokens;
    p.D = dim;
    p.F = hidden;
    const MlpSpace fwd(p, bf16, false), bwd(p, bf16, true);
    for (const ProductPlan& q : {is_skinny(p, bf16) ? ProductPlan{-1, 1} : fwd.gate, bwd.gate,
                                 bwd.input, bwd.weights}) {
        *tiles++ = q.tile;
        *tiles++ = q.splits;
    }
}

hipError_t launch_mlp_fwd(const MlpParams& p, bool bf16, hipStream_t stream) {
    return bf16 ? forward<bf16_t>(p, stream) : forward<float>(p, stream);
}

hipError_t launch_mlp_bwd(const MlpParams& p, bool bf16, hipStream_t stream) {
    return bf16 ? backward<bf16_t>(p, stream) : backward<float>(p, stream);
}

MSEL_BOUNDS_TAKER(take_bounds_mlp)

}  // namespace msel
