// gated_mlp.hip -- the gated feed-forward block out = act(x Wg^T) * (x Wu^T) and its backward
//   dG = dout U act'(G), dU = dout act(G);  dx = dG Wg + dU Wu;  dWg = dG^T x, dWu = dU^T x
// as MFMA products of rows with consecutive k: C[m][n] = sum_k A[m][k] B[n][k].
//
// The matrix cores bound it.  A block computes a tile of C with both operands staged in LDS, one
// stage of 128 bytes of k ahead, loaded without a register between (global_load_lds).  A row of a
// stage is 8 chunks of 16 bytes, chunk c of row r at place c ^ (r & 7): the 8 lanes that LDS serves
// together read one chunk of 8 rows, which then lie in 8 different places.  In the fused product the
// B rows of a wavefront are 32 rows of Wg and the same 32 of Wu, so that a lane holds G and U of the
// same elements and the activation and the product need no exchange.
// The MFMA's rows are C's columns: a lane then holds 4 consecutive columns of a row of C.
//
// Operands whose rows are no multiple of a stage are copied into padded rows first; the backward's
// products over the hidden width and over the tokens read transposed copies.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block_kernels.hpp"
#include "lm_device.hpp"

namespace msel {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kStageBytes = 128;  // of k per stage
constexpr int kSteps = kStageBytes / 32;

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
    if constexpr (!GELU) return silu_f(z);
    return z * sigmoid_f(kTwoC * z * fmaf(0.044715f * z, z, 1.0f));
}
template <bool GELU>
__device__ __forceinline__ void act_grad(float z, float& v, float& slope) {
    if constexpr (!GELU) {
        silu_grad_f(z, v, slope);
    } else {
        const float s = sigmoid_f(kTwoC * z * fmaf(0.044715f * z, z, 1.0f));
        v = z * s;
        slope = fmaf(v * (1.0f - s), kTwoC * fmaf(0.134145f * z, z, 1.0f), s);
    }
}

enum class Epi { kPlain, kGate, kGateGrad };

struct ProductParams {
    int64_t M;       // rows of A and C
    int N;           // kPlain: rows of B; else the hidden width (rows of each weight)
    int64_t K;       // a multiple of a stage
    const void* a;   // [M, lda]
    const void* b0;  // [N, ldb]
    const void* b1;  // the other weight
    int64_t lda, ldb;
    void* c0;        // rows below `split`
    void* c1;        // rows from `split` on (kPlain)
    int64_t split, ldc;
    const void* dout;  // kGateGrad: [M, N]
    int hp;            // kGateGrad: dG in columns [0, hp) of C, dU in [hp, 2 hp)
    int tm, tn;        // tiles
};

// The tile of a block: consecutive tiles on one XCD, in bands of 8 tiles of rows, so that the
// blocks that run together share rows of both operands in its L2.
__device__ __forceinline__ bool tile_at(const ProductParams& p, int& m, int& n) {
    const int64_t tiles = static_cast<int64_t>(p.tm) * p.tn;
    const int64_t bid = blockIdx.y * static_cast<int64_t>(gridDim.x) + blockIdx.x;
    if (bid >= tiles) return false;
    const int id = gridDim.y == 1 ? static_cast<int>(xcd_order(blockIdx.x, gridDim.x))
                                  : static_cast<int>(bid);
    constexpr int kBand = 8;
    const int width = kBand * p.tn;
    const int band = id / width, in = id - band * width;
    const int rows = min(kBand, p.tm - band * kBand);
    m = band * kBand + in % rows;
    n = in / rows;
    return true;
}

// 4 values into columns [col, col + 4) of a row of n columns.
template <typename T>
__device__ __forceinline__ void store4(T* row, int col, int n, const float (&v)[4]) {
    if (col + 4 <= n) {
        if constexpr (sizeof(T) == 4) {
            st_vec<float, 4>(row + MSEL_SPAN(col, 4, n), v);
        } else {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            const u32x2 w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            __builtin_memcpy(row + MSEL_SPAN(col, 4, n), &w, 8);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (col + k < n) Elem<T>::store1(row + col + k, v[k]);
}

template <typename T>
__device__ __forceinline__ void load4(const T* row, int col, int n, float (&v)[4]) {
    if (col + 4 <= n) {
        if constexpr (sizeof(T) == 4) {
            to_f32<float, 4>(ld_raw<float, 4>(row + MSEL_SPAN(col, 4, n)), v);
        } else {
            uint32_t w[2];
            __builtin_memcpy(w, row + MSEL_SPAN(col, 4, n), 8);
            v[0] = bf16lo(w[0]);
            v[1] = bf16hi(w[0]);
            v[2] = bf16lo(w[1]);
            v[3] = bf16hi(w[1]);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = col + k < n ? Elem<T>::load1(row + col + k) : 0.0f;
}

typedef __attribute__((address_space(1))) const void GlobalVoid;
typedef __attribute__((address_space(3))) void LdsVoid;

// WM x WN wavefronts, each MI x 2 MFMA tiles of 32 x 32: a block computes WM MI 32 rows by
// WN 64 rows of B (in the fused products WN 32 columns of both weights).
template <typename T, int WM, int WN, int MI, Epi EPI, bool GELU>
__global__ __launch_bounds__(WM* WN * 64, 2) void product_kernel(ProductParams p) {
    constexpr int kThreads = WM * WN * 64;
    constexpr int BM = WM * MI * 32, BN = WN * 64;
    constexpr int kRound = kThreads / 8;  // rows that the block loads at once
    constexpr int LA = BM / kRound, LB = BN / kRound;
    constexpr bool kDual = EPI != Epi::kPlain;
    constexpr int kStage = (BM + BN) * kStageBytes;
    static_assert(BM % kRound == 0 && BN % kRound == 0, "whole rounds");
    extern __shared__ __align__(16) char lds[];

    int tile_m, tile_n;
    if (!tile_at(p, tile_m, tile_n)) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = lane_id();
    const int wm = wave / WN, wn = wave % WN;
    const int64_t m0 = static_cast<int64_t>(tile_m) * BM;
    const int n0 = tile_n * (kDual ? BN / 2 : BN);

    // this thread's chunks of a stage: row r of a round, place tid % 8; rows past the end repeat
    // the last one (their results are not stored)
    const char* src[LA + LB];
#pragma unroll
    for (int i = 0; i < LA + LB; ++i) {
        const int r = (i < LA ? i : i - LA) * kRound + (tid >> 3);
        const int chunk = (tid & 7) ^ (r & 7);
        const T* row;
        if (i < LA) {
            const int64_t m = min(m0 + r, p.M - 1);
            row = static_cast<const T*>(p.a) + MSEL_IDX(m, p.M) * p.lda;
        } else if (kDual) {
            const int n = min(n0 + (r >> 6) * 32 + (r & 31), p.N - 1);
            row = static_cast<const T*>((r & 32) ? p.b1 : p.b0) +
                  static_cast<int64_t>(MSEL_IDX(n, p.N)) * p.ldb;
        } else {
            const int n = min(n0 + r, p.N - 1);
            row = static_cast<const T*>(p.b0) + static_cast<int64_t>(MSEL_IDX(n, p.N)) * p.ldb;
        }
        src[i] = reinterpret_cast<const char*>(row) + chunk * 16;
    }
    const auto load_stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < LA + LB; ++i) {
            const int at = buf * kStage + (i * kThreads + wave * 64) * 16;
            __builtin_amdgcn_global_load_lds((GlobalVoid*)src[i], (LdsVoid*)(lds + at), 16, 0, 0);
            src[i] += kStageBytes;
        }
    };

    f32x16 acc[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    const int row_a = wm * MI * 32 + (lane & 31), row_b = wn * 64 + (lane & 31);
    const int stages = static_cast<int>(p.K / kStageK<T>);
    load_stage(0);
    for (int k = 0; k < stages; ++k) {
        __syncthreads();  // the stage has landed, and the other buffer has been read
        if (k + 1 < stages) load_stage((k + 1) & 1);
        const char* sa = lds + (k & 1) * kStage;
        const char* sb = sa + BM * kStageBytes;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int c = 2 * s + (lane >> 5);
            u32x4 fa[MI], fb[2];
#pragma unroll
            for (int i = 0; i < MI; ++i)
                fa[i] = *reinterpret_cast<const u32x4*>(sa + (row_a + i * 32) * kStageBytes +
                                                        ((c ^ (lane & 7)) * 16));
#pragma unroll
            for (int j = 0; j < 2; ++j)
                fb[j] = *reinterpret_cast<const u32x4*>(sb + (row_b + j * 32) * kStageBytes +
                                                        ((c ^ (lane & 7)) * 16));
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    mfma_step(static_cast<const T*>(nullptr), fb[j], fa[i], acc[i][j]);
        }
    }

    // D: lane l holds column l % 32 (a row of C) and rows 8 g + 4 (l / 32) + 0..3 (columns of C)
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t m = m0 + wm * MI * 32 + i * 32 + (lane & 31);
        if (m >= p.M) continue;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int in = 8 * g + 4 * (lane >> 5);
            if constexpr (EPI == Epi::kPlain) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int n = n0 + wn * 64 + j * 32 + in;
                    T* row = m < p.split ? static_cast<T*>(p.c0) + m * p.ldc
                                         : static_cast<T*>(p.c1) + (m - p.split) * p.ldc;
                    const float v[4] = {acc[i][j][4 * g], acc[i][j][4 * g + 1],
                                        acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                    store4(row, n, p.N, v);
                }
            } else if constexpr (EPI == Epi::kGate) {
                const int n = n0 + wn * 32 + in;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = act_of<GELU>(acc[i][0][4 * g + e]) * acc[i][1][4 * g + e];
                store4(static_cast<T*>(p.c0) + m * p.ldc, n, p.N, v);
            } else {
                const int n = n0 + wn * 32 + in;
                float d[4], dg[4], du[4];
                load4(static_cast<const T*>(p.dout) + m * p.N, n, p.N, d);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v, slope;
                    act_grad<GELU>(acc[i][0][4 * g + e], v, slope);
                    // columns behind the weights' last row are 0: the next product reads them
                    dg[e] = n + e < p.N ? d[e] * acc[i][1][4 * g + e] * slope : 0.0f;
                    du[e] = n + e < p.N ? d[e] * v : 0.0f;
                }
                T* row = static_cast<T*>(p.c0) + m * p.ldc;
                store4(row, n, p.hp, dg);
                store4(row + p.hp, n, p.hp, du);
            }
        }
    }
}

// dst[r][c] = src[r][c] for c < cols, 0 up to ldd.
template <typename T>
__global__ __launch_bounds__(256) void pad_kernel(const T* src, int64_t rows, int64_t cols, T* dst,
                                                  int64_t ldd) {
    const int64_t n = rows * ldd;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = i / ldd, c = i - r * ldd;
        const float v = c < cols ? Elem<T>::load1(src + MSEL_IDX(r * cols + c, rows * cols)) : 0.0f;
        Elem<T>::store1(dst + MSEL_IDX(i, n), v);
    }
}

// dst[c][r] = src[r][c] for r < rows, 0 up to fill (<= ldd), over tiles of 64 x 64.
template <typename T>
__global__ __launch_bounds__(256) void transpose_kernel(const T* src, int64_t rows, int64_t cols,
                                                        int64_t lds_, T* dst, int64_t ldd,
                                                        int64_t fill) {
    __shared__ T tile[64][66];
    const int64_t tr = (fill + 63) / 64, tc = (cols + 63) / 64;
    for (int64_t t = blockIdx.x; t < tr * tc; t += gridDim.x) {
        const int64_t r0 = t % tr * 64, c0 = t / tr * 64;
        const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
#pragma unroll 4
        for (int k = y; k < 64; k += 4) {
            T v{};
            if (r0 + k < rows && c0 + x < cols)
                v = src[MSEL_IDX((r0 + k) * lds_ + c0 + x, (rows - 1) * lds_ + cols)];
            tile[k][x] = v;
        }
        __syncthreads();
#pragma unroll 4
        for (int k = y; k < 64; k += 4)
            if (c0 + k < cols && r0 + x < fill)
                dst[MSEL_IDX((c0 + k) * ldd + r0 + x, (cols - 1) * ldd + fill)] = tile[x][k];
        __syncthreads();
    }
}

constexpr unsigned kMaxBlocks = 1u << 20;

template <typename T>
void pad(const void* src, int64_t rows, int64_t cols, void* dst, int64_t ldd, hipStream_t stream) {
    const int64_t blocks = (rows * ldd + 1023) / 1024;
    hipLaunchKernelGGL(pad_kernel<T>,
                       dim3(static_cast<unsigned>(std::min<int64_t>(blocks, kMaxBlocks))),
                       dim3(256), 0, stream, static_cast<const T*>(src), rows, cols,
                       static_cast<T*>(dst), ldd);
}

template <typename T>
void transpose(const void* src, int64_t rows, int64_t cols, int64_t lds_, void* dst, int64_t ldd,
               int64_t fill, hipStream_t stream) {
    const int64_t tiles = (fill + 63) / 64 * ((cols + 63) / 64);
    hipLaunchKernelGGL(transpose_kernel<T>,
                       dim3(static_cast<unsigned>(std::min<int64_t>(tiles, kMaxBlocks))),
                       dim3(256), 0, stream, static_cast<const T*>(src), rows, cols, lds_,
                       static_cast<T*>(dst), ldd, fill);
}

template <typename T, int WM, int WN, int MI, Epi EPI, bool GELU>
hipError_t launch_tiles(ProductParams p, hipStream_t stream) {
    constexpr int BM = WM * MI * 32, BN = WN * 64;
    constexpr int bytes = 2 * (BM + BN) * kStageBytes;
    const int bn = EPI == Epi::kPlain ? BN : BN / 2;
    p.tm = static_cast<int>((p.M + BM - 1) / BM);
    const int cols = EPI == Epi::kGateGrad ? p.hp : p.N;
    p.tn = (cols + bn - 1) / bn;
    const hipError_t e = allow_dynamic_lds<product_kernel<T, WM, WN, MI, EPI, GELU>>(bytes);
    if (e != hipSuccess) return e;
    const int64_t tiles = static_cast<int64_t>(p.tm) * p.tn;
    const dim3 grid = tiles <= kMaxBlocks
                          ? dim3(static_cast<unsigned>(tiles))
                          : dim3(kMaxBlocks, static_cast<unsigned>((tiles + kMaxBlocks - 1) / kMaxBlocks));
    hipLaunchKernelGGL((product_kernel<T, WM, WN, MI, EPI, GELU>), grid, dim3(WM * WN * 64), bytes,
                       stream, p);
    return hipGetLastError();
}

// Tiles of 256 x 256 where they fill the chip, else of 128 x 128.
template <typename T, Epi EPI, bool GELU>
hipError_t launch_product(const ProductParams& p, hipStream_t stream) {
    const int64_t cols = EPI == Epi::kPlain ? p.N : 2 * static_cast<int64_t>(p.N);
    const int64_t wide = (p.M + 255) / 256 * ((cols + 255) / 256);
    if (wide >= 256) return launch_tiles<T, 2, 4, 4, EPI, GELU>(p, stream);
    return launch_tiles<T, 2, 2, 2, EPI, GELU>(p, stream);
}

// ---- workspaces --------------------------------------------------------------------------------

int64_t up_to(int64_t n, int64_t q) { return (n + q - 1) / q * q; }

// Offsets in bytes; absent parts take none.
struct MlpSpace {
    int64_t dp, hp, mp;  // padded width, hidden width, tokens
    size_t x = 0, wg = 0, wu = 0, wt = 0, dgu = 0, dgu_t = 0, x_t = 0, all = 0;
    MlpSpace(const MlpParams& p, size_t elem, bool bwd) {
        const int64_t q = kStageBytes / static_cast<int64_t>(elem);
        dp = up_to(p.D, q);
        hp = up_to(p.F, q);
        mp = up_to(p.M, q);
        const auto take = [&](int64_t elems) {
            const size_t at = all;
            all += (static_cast<size_t>(elems) * elem + 255) / 256 * 256;
            return at;
        };
        if (dp != p.D) {
            x = take(p.M * dp);
            wg = take(p.F * dp);
            wu = take(p.F * dp);
        }
        if (!bwd) return;
        dgu = take(p.M * 2 * hp);
        wt = take(p.D * 2 * hp);
        dgu_t = take(2 * p.F * mp);
        x_t = take(p.D * mp);
    }
};

template <typename T, bool GELU>
hipError_t gate(const MlpParams& p, const MlpSpace& w, bool grad, hipStream_t stream) {
    char* const ws = static_cast<char*>(p.ws);
    ProductParams q{};
    q.M = p.M;
    q.N = p.F;
    q.K = w.dp;
    q.lda = q.ldb = w.dp;
    q.a = p.x;
    q.b0 = p.wg;
    q.b1 = p.wu;
    if (w.dp != p.D) {
        pad<T>(p.x, p.M, p.D, ws + w.x, w.dp, stream);
        pad<T>(p.wg, p.F, p.D, ws + w.wg, w.dp, stream);
        pad<T>(p.wu, p.F, p.D, ws + w.wu, w.dp, stream);
        q.a = ws + w.x;
        q.b0 = ws + w.wg;
        q.b1 = ws + w.wu;
    }
    if (!grad) {
        q.c0 = p.out;
        q.ldc = p.F;
        return launch_product<T, Epi::kGate, GELU>(q, stream);
    }
    q.c0 = ws + w.dgu;
    q.ldc = 2 * w.hp;
    q.hp = static_cast<int>(w.hp);
    q.dout = p.dout;
    return launch_product<T, Epi::kGateGrad, GELU>(q, stream);
}

template <typename T>
hipError_t backward(const MlpParams& p, hipStream_t stream) {
    const MlpSpace w(p, sizeof(T), true);
    char* const ws = static_cast<char*>(p.ws);
    hipError_t e = p.gelu ? gate<T, true>(p, w, true, stream) : gate<T, false>(p, w, true, stream);
    if (e != hipSuccess) return e;
    if (p.dx != nullptr) {  // dx[m][d] = sum over 2 hp of dgu[m] wt[d]
        T* const wt = reinterpret_cast<T*>(ws + w.wt);
        transpose<T>(p.wg, p.F, p.D, p.D, wt, 2 * w.hp, w.hp, stream);
        transpose<T>(p.wu, p.F, p.D, p.D, wt + w.hp, 2 * w.hp, w.hp, stream);
        ProductParams q{};
        q.M = q.split = p.M;
        q.N = p.D;
        q.K = q.lda = q.ldb = 2 * w.hp;
        q.a = ws + w.dgu;
        q.b0 = wt;
        q.c0 = p.dx;
        q.ldc = p.D;
        e = launch_product<T, Epi::kPlain, false>(q, stream);
        if (e != hipSuccess) return e;
    }
    if (p.dwg != nullptr) {  // dw[f][d] = sum over tokens of dgu_t[f] x_t[d]
        T* const gt = reinterpret_cast<T*>(ws + w.dgu_t);
        const T* const dgu = reinterpret_cast<const T*>(ws + w.dgu);
        transpose<T>(dgu, p.M, p.F, 2 * w.hp, gt, w.mp, w.mp, stream);
        transpose<T>(dgu + w.hp, p.M, p.F, 2 * w.hp, gt + p.F * w.mp, w.mp, w.mp, stream);
        transpose<T>(p.x, p.M, p.D, p.D, ws + w.x_t, w.mp, w.mp, stream);
        ProductParams q{};
        q.M = 2 * static_cast<int64_t>(p.F);
        q.split = p.F;
        q.N = p.D;
        q.K = q.lda = q.ldb = w.mp;
        q.a = gt;
        q.b0 = ws + w.x_t;
        q.c0 = p.dwg;
        q.c1 = p.dwu;
        q.ldc = p.D;
        e = launch_product<T, Epi::kPlain, false>(q, stream);
    }
    return e;
}

template <typename T>
hipError_t forward(const MlpParams& p, hipStream_t stream) {
    const MlpSpace w(p, sizeof(T), false);
    return p.gelu ? gate<T, true>(p, w, false, stream) : gate<T, false>(p, w, false, stream);
}

}  // namespace

size_t mlp_fwd_workspace_bytes(const MlpParams& p, bool bf16) {
    return MlpSpace(p, bf16 ? 2 : 4, false).all;
}

size_t mlp_bwd_workspace_bytes(const MlpParams& p, bool bf16) {
    return MlpSpace(p, bf16 ? 2 : 4, true).all;
}

hipError_t launch_mlp_fwd(const MlpParams& p, bool bf16, hipStream_t stream) {
    return bf16 ? forward<bf16_t>(p, stream) : forward<float>(p, stream);
}

hipError_t launch_mlp_bwd(const MlpParams& p, bool bf16, hipStream_t stream) {
    return bf16 ? backward<bf16_t>(p, stream) : backward<float>(p, stream);
}

MSEL_BOUNDS_TAKER(take_bounds_mlp)

}  // namespace msel
