// lm_kernels.hpp -- internal interface between the C ABI of the operators around the scan
// (lm_api.cpp) and their kernels: the norms, the embedding, the gradient norm and clipping.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "msel_kernels.hpp"

namespace msel {

constexpr int kMaxNormDim = 16384;  // the boundary's MSEL_MAX_NORM_DIM

enum class NormMode { kResidual, kGateFirst, kGateLast };

// A norm over contiguous rows: `rows` tokens of `groups` groups of n values each; row (r, g)
// starts at element (r * groups + g) * n and takes its weights from w + g * n.
// kResidual: a is x (forward) or s (backward), b the residual or dresidual_out (may be null);
// the gated modes: a is x, b is z.
struct RowNormParams {
    int64_t rows;
    int groups, n;
    float scale, eps;
    const void* a;
    const void* b;
    const float* w;
    const void* dout;
    void* out;       // forward: out; backward: dx
    void* out2;      // forward: residual_out; backward: dresidual, or dz
    float* dw_part;  // backward: [blocks][groups * n] partial sums, or null
    float* dw;       // backward: [groups * n], or null
};
// Rows of partial dweight sums that a backward over these sizes writes.
int row_norm_partials(int64_t rows, int groups, int n, NormMode mode, bool bf16, bool rbf16);
hipError_t launch_row_norm_fwd(const RowNormParams& p, NormMode mode, bool bf16, bool rbf16,
                               hipStream_t stream);
hipError_t launch_row_norm_bwd(const RowNormParams& p, NormMode mode, bool bf16, bool rbf16,
                               hipStream_t stream);

// dw[c] = sum over r of part[r][c], r in order: part is [rows][cols].
hipError_t launch_column_sums(float* part, int64_t rows, int64_t cols, float* dw,
                              hipStream_t stream);

// The gated norm over the channels of [batch, D, L]; out_bld: out and dout are [batch, L, D].
struct TileNormParams {
    int B, D, L, groups, n;  // n = D / groups
    int tiles;               // token tiles per batch row, set by the launchers
    float eps;
    int out_bld;
    const void* x;
    const void* z;
    const float* w;
    const void* dout;
    void* out;       // forward: out; backward: dx
    void* dz;
    float* dw_part;  // backward: [tiles of all batch rows][D] partial sums, or null
    float* dw;
};
// Rows of partial dweight sums that a backward over these sizes may write.
int64_t tile_norm_partials(int B, int groups, int n, int L, bool bf16);
// Whether the launch goes to the kernels for few or short tiles (tile_short.hip), and else the
// bytes of a channel's row in its narrowest tiles.
bool tile_is_short(int B, int groups, int L, bool bf16);
int narrow_bytes(int B, int groups, int n, int L, bool bf16);
int64_t tile_short_partials(int B, int groups, int L);
hipError_t launch_tile_short(const TileNormParams& p, bool gate_first, bool bf16, bool bwd,
                             hipStream_t stream);
hipError_t launch_tile_norm_fwd(const TileNormParams& p, bool gate_first, bool bf16,
                                hipStream_t stream);
hipError_t launch_tile_norm_bwd(const TileNormParams& p, bool gate_first, bool bf16,
                                hipStream_t stream);

struct EmbedParams {
    int64_t tokens;
    int vocab, dim;
    int ids64;
    int64_t padding_idx;
    float scale;
    const void* ids;
    const void* w;
    void* out;
    const void* dout;
    const float* base;
    float* dw;
    void* ws;
};
size_t embed_workspace_bytes(int64_t tokens, int vocab, int dim);
hipError_t launch_embed_fwd(const EmbedParams& p, bool wbf16, bool bf16, hipStream_t stream);
hipError_t launch_embed_bwd(const EmbedParams& p, bool bf16, hipStream_t stream);

struct GradTensor {
    const void* src;
    void* dst;
    int64_t n;
    bool bf16;
};
// A reader of the caller's tensor list: entry i (i < count).
using GradReader = GradTensor (*)(const void* list, const void* outs, int i);
struct GradNormParams {
    int count;
    const void* list;
    const void* outs;
    GradReader read;
    float max_norm, eps;
    float* norm;
    double* partials;
};
// Partial sums (one double each) of a list of these tensors.
int64_t grad_partials(const GradNormParams& p);
// norm; with clip, also the scaled tensors.
hipError_t launch_grad_norm(const GradNormParams& p, bool clip, hipStream_t stream);

hipError_t take_bounds_row_norm(BoundsRecord* r);
hipError_t take_bounds_tile_norm(BoundsRecord* r);
hipError_t take_bounds_tile_norm_bwd(BoundsRecord* r);
hipError_t take_bounds_tile_short(BoundsRecord* r);
hipError_t take_bounds_embed(BoundsRecord* r);
hipError_t take_bounds_grads(BoundsRecord* r);

}  // namespace msel
