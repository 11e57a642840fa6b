// block_kernels.hpp -- internal interface between the C ABI (block_api.cpp) and the kernels of the
// gated linear recurrence, the gated feed-forward block and the log probabilities of tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "msel_kernels.hpp"

namespace msel {

// ---- the gated linear recurrence -----------------------------------------------------------

struct LruParams {
    int B, D, L, nchunks;
    const void* x;
    const void* ga;
    const void* gx;
    const float* lam;
    const float* h0;
    void* out;           // forward: null in a pass for the states alone
    float* final_state;
    float* chunks;       // [B, D, nchunks]: forward: written unless null; backward: read
    float2* pairs;       // [B * D, nseg + 1]: the segments' compositions (plans of several
                         // segments); forward: behind an entry for h0
    const void* dout;
    const float* dfinal;
    void* dx;
    void* dga;
    void* dgx;
    float* dh0;
    float* dlam_part;    // [B * nseg, D], or null (dlam itself where that is one part)
    float* dlam;
    int nseg, seg_tiles; // set by the launchers
};
// How a row is worked on: `team` lanes per row, or a wavefront per segment of seg_tiles tiles.
struct LruPlan {
    int team, tiles, nseg, seg_tiles;
};
LruPlan lru_plan(int64_t rows, int L, bool bwd);
hipError_t launch_lru_fwd(const LruParams& p, bool bf16, hipStream_t stream);
hipError_t launch_lru_bwd(const LruParams& p, bool bf16, hipStream_t stream);

// ---- log probabilities ---------------------------------------------------------------------

constexpr int kMaxTop = 64;  // the boundary's MSEL_MAX_TOP

struct LogprobParams {
    int64_t rows, stride, dstride;  // elements from a row to the next
    int V, ids64, top;
    float scale;
    const void* logits;
    const void* ids;       // null: no token asked for
    float* logprob;
    float* lse;
    float* entropy;
    int64_t* top_ids;      // [rows, top]
    float* top_logprobs;
    void* ws;              // parts of rows that several blocks share
    const float* in_lse;
    const float* in_entropy;
    const float* dlogprob;
    const float* dlse;
    const float* dentropy;
    void* dlogits;
    int slices;            // set by the launchers
    int slice;             // columns of a slice
};
size_t logprob_workspace_bytes(int64_t rows, int V, int top, bool bf16);
hipError_t launch_logprob_fwd(const LogprobParams& p, bool bf16, hipStream_t stream);
hipError_t launch_logprob_bwd(const LogprobParams& p, bool bf16, hipStream_t stream);

// ---- the gated feed-forward block ----------------------------------------------------------

struct MlpParams {
    int64_t M;             // tokens
    int D, F;              // width, hidden width
    int gelu;              // 0: silu; 1: gelu, tanh form
    const void* x;
    const void* wg;
    const void* wu;
    void* out;
    const void* dout;
    void* dx;
    void* dwg;
    void* dwu;
    void* ws;
};
size_t mlp_fwd_workspace_bytes(const MlpParams& p, bool bf16);
size_t mlp_bwd_workspace_bytes(const MlpParams& p, bool bf16);
// Which kernels a call takes, for the tests' choice of sizes: the tile (0: 256 x 256, 1: 128 x 128,
// 2: 64 x 128, -1: none, the kernel for few tokens) and the splits of the forward's product, then
// of the backward's three (dG and dU, dx, the weights' gradients).  8 ints.
void mlp_tiles(int64_t tokens, int dim, int hidden, bool bf16, int* tiles);
hipError_t launch_mlp_fwd(const MlpParams& p, bool bf16, hipStream_t stream);
hipError_t launch_mlp_bwd(const MlpParams& p, bool bf16, hipStream_t stream);

hipError_t take_bounds_lru(BoundsRecord* r);
hipError_t take_bounds_logprob(BoundsRecord* r);
hipError_t take_bounds_mlp(BoundsRecord* r);

}  // namespace msel
