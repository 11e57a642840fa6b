// block_api.cpp -- the extern "C" entry points of the gated linear recurrence, the log
// probabilities of tokens and the gated feed-forward block, declared in include/msel.h.
//
// As in msel_api.cpp, every entry point validates its arguments on the host (no HIP call, no
// device memory touched) and only then enqueues kernels on the caller's stream; no device memory
// is allocated, and nothing is kept between calls or synchronized.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "block_kernels.hpp"
#include "msel.h"

static_assert(MSEL_MAX_TOP == msel::kMaxTop, "the kernels' limit is the boundary's");

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxChannels = int64_t(1) << 27;  // dlam's sum: 64 of them per block of 1024

typedef std::initializer_list<const void*> Pointers;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool is_dtype(int32_t d) { return d == MSEL_F32 || d == MSEL_BF16; }
bool is_flag(int32_t f) { return f == 0 || f == 1; }
msel_status hip_status(hipError_t e) { return e == hipSuccess ? MSEL_OK : MSEL_ERR_HIP; }
uintptr_t elem_bytes(int32_t dtype) { return dtype == MSEL_BF16 ? 2 : 4; }

bool any_null(Pointers ps) { return std::find(ps.begin(), ps.end(), nullptr) != ps.end(); }
bool all_aligned(Pointers ps, uintptr_t a) {
    return std::all_of(ps.begin(), ps.end(), [=](const void* p) { return aligned(p, a); });
}

// The memory that an argument names (none for a null or an empty one).
struct Memory {
    uintptr_t from = 0, to = 0;
    Memory(const void* p, uint64_t bytes)
        : from(reinterpret_cast<uintptr_t>(p)), to(p == nullptr || bytes == 0 ? 0 : from + bytes) {}
    bool meets(const Memory& o) const { return from < o.to && o.from < to; }
};
typedef std::initializer_list<Memory> Memories;

// Whether an output shares memory with an input or another output.
bool aliased(Memories outs, Memories ins) {
    for (const Memory* o = outs.begin(); o != outs.end(); ++o) {
        const auto met = [o](const Memory& m) { return o->meets(m); };
        if (std::any_of(ins.begin(), ins.end(), met) || std::any_of(outs.begin(), o, met))
            return true;
    }
    return false;
}

// Of a workspace that shares memory with none of `others`.
msel_status check_workspace(const void* ws, size_t have, size_t need, Memories others) {
    if (need == 0) return MSEL_OK;
    if (ws == nullptr || have < need) return MSEL_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return MSEL_ERR_ALIGN;
    return aliased({{ws, need}}, others) ? MSEL_ERR_ALIAS : MSEL_OK;
}

size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }

// ---- the gated linear recurrence -----------------------------------------------------------

msel_status check_lru_sizes(const msel_lru_args* a) {
    if (a == nullptr) return MSEL_ERR_NULL;
    if (a->abi_version != MSEL_ABI_VERSION || a->reserved != 0) return MSEL_ERR_VERSION;
    if (a->batch < 1 || a->dim < 1 || a->seqlen < 1) return MSEL_ERR_SHAPE;
    const int64_t rows = static_cast<int64_t>(a->batch) * a->dim;
    if (a->seqlen > MSEL_MAX_SEQLEN || a->dim > kMaxChannels || rows > kMaxRows ||
        rows > kMaxElems / a->seqlen)
        return MSEL_ERR_SHAPE;
    return is_dtype(a->dtype) ? MSEL_OK : MSEL_ERR_DTYPE;
}

msel_status check_lru(const msel_lru_args* a) {
    const msel_status s = check_lru_sizes(a);
    if (s != MSEL_OK) return s;
    if (any_null({a->x, a->gate_a, a->gate_x, a->lam})) return MSEL_ERR_NULL;
    if (!all_aligned({a->x, a->gate_a, a->gate_x}, 16) ||
        !all_aligned({a->lam, a->h0, a->chunk_states}, 4))
        return MSEL_ERR_ALIGN;
    return MSEL_OK;
}

// Bytes of the recurrence's tensors.
struct LruBytes {
    uint64_t act, lam, state, chunks;
    explicit LruBytes(const msel_lru_args* a) {
        const uint64_t rows = static_cast<uint64_t>(a->batch) * static_cast<uint64_t>(a->dim);
        act = rows * static_cast<uint64_t>(a->seqlen) * elem_bytes(a->dtype);
        lam = static_cast<uint64_t>(a->dim) * 4;
        state = rows * 4;
        chunks = rows * static_cast<uint64_t>(msel_num_chunks(a->seqlen)) * 4;
    }
};

// The parts of a workspace, in the order in which they lie.
struct LruSpace {
    size_t pairs = 0, chunks = 0, dlam = 0;  // bytes
    size_t all() const { return rounded(pairs) + rounded(chunks) + rounded(dlam); }
};

LruSpace lru_space(const msel_lru_args* a, bool bwd) {
    const size_t rows = static_cast<size_t>(a->batch) * static_cast<size_t>(a->dim);
    const msel::LruPlan q = msel::lru_plan(static_cast<int64_t>(rows), a->seqlen, bwd);
    LruSpace w;
    // both directions cut the same rows into the same segments
    if (q.nseg > 1) w.pairs = rows * static_cast<size_t>(q.nseg + 1) * sizeof(float2);
    if (!bwd) return w;
    // rows of up to a chunk start from h0
    if (a->chunk_states == nullptr && q.team >= 64)
        w.chunks = rows * static_cast<size_t>(msel_num_chunks(a->seqlen)) * sizeof(float);
    w.dlam = rows * static_cast<size_t>(q.nseg) * sizeof(float);
    return w;
}

msel::LruParams lru_params(const msel_lru_args* a) {
    msel::LruParams p{};
    p.B = a->batch;
    p.D = a->dim;
    p.L = a->seqlen;
    p.nchunks = msel_num_chunks(a->seqlen);
    p.x = a->x;
    p.ga = a->gate_a;
    p.gx = a->gate_x;
    p.lam = a->lam;
    p.h0 = a->h0;
    return p;
}

// ---- log probabilities ---------------------------------------------------------------------

msel_status check_logprob(const msel_logprob_args* a) {
    if (a == nullptr) return MSEL_ERR_NULL;
    if (a->abi_version != MSEL_ABI_VERSION) return MSEL_ERR_VERSION;
    if (a->vocab < 1 || a->vocab > kMaxRows || a->rows < 1 || a->rows > kMaxRows ||
        a->stride < a->vocab || a->stride > kMaxElems / a->rows)
        return MSEL_ERR_SHAPE;
    if (!is_dtype(a->dtype) || !is_flag(a->ids_64bit)) return MSEL_ERR_DTYPE;
    if (!(a->scale > 0.0f) || !isfinite(a->scale)) return MSEL_ERR_SHAPE;
    return MSEL_OK;
}

bool logprob_aligned(const msel_logprob_args* a) {
    return aligned(a->logits, elem_bytes(a->dtype)) && aligned(a->ids, a->ids_64bit ? 8 : 4) &&
           all_aligned({a->logprob, a->lse, a->entropy, a->top_logprobs}, 4) &&
           aligned(a->top_ids, 8);
}

// From the first logit of strided rows to the last, a value per row, and the ids.
Memory logits_at(const msel_logprob_args* a, const void* p, int64_t stride) {
    return {p, static_cast<uint64_t>((a->rows - 1) * stride + a->vocab) * elem_bytes(a->dtype)};
}
Memory rows_at(const msel_logprob_args* a, const void* p) {
    return {p, static_cast<uint64_t>(a->rows) * 4};
}
Memory ids_at(const msel_logprob_args* a) {
    return {a->ids, static_cast<uint64_t>(a->rows) * (a->ids_64bit ? 8 : 4)};
}

size_t logprob_ws(const msel_logprob_args* a) {
    return msel::logprob_workspace_bytes(a->rows, a->vocab, a->top, a->dtype == MSEL_BF16);
}

msel::LogprobParams logprob_params(const msel_logprob_args* a) {
    msel::LogprobParams p{};
    p.rows = a->rows;
    p.stride = a->stride;
    p.V = a->vocab;
    p.ids64 = a->ids_64bit;
    p.scale = a->scale;
    p.logits = a->logits;
    p.ids = a->ids;
    return p;
}

// ---- the gated feed-forward block ----------------------------------------------------------

msel_status check_mlp_sizes(const msel_gated_mlp_args* a) {
    if (a == nullptr) return MSEL_ERR_NULL;
    if (a->abi_version != MSEL_ABI_VERSION || a->reserved != 0) return MSEL_ERR_VERSION;
    if (a->dim < 1 || a->hidden < 1 || a->tokens < 1 || a->tokens > (int64_t(1) << 24))
        return MSEL_ERR_SHAPE;
    if (a->dim > MSEL_MAX_MLP_WIDTH || a->hidden > MSEL_MAX_MLP_WIDTH) return MSEL_ERR_UNSUPPORTED;
    if (a->tokens > kMaxElems / std::max(a->dim, a->hidden)) return MSEL_ERR_SHAPE;
    return is_dtype(a->dtype) && is_flag(a->activation) ? MSEL_OK : MSEL_ERR_DTYPE;
}

msel_status check_mlp(const msel_gated_mlp_args* a) {
    const msel_status s = check_mlp_sizes(a);
    if (s != MSEL_OK) return s;
    if (any_null({a->x, a->w_gate, a->w_up})) return MSEL_ERR_NULL;
    return all_aligned({a->x, a->w_gate, a->w_up}, 16) ? MSEL_OK : MSEL_ERR_ALIGN;
}

// Bytes of the block's tensors.
struct MlpBytes {
    uint64_t x, w, out;
    explicit MlpBytes(const msel_gated_mlp_args* a) {
        const uint64_t e = elem_bytes(a->dtype), m = static_cast<uint64_t>(a->tokens);
        x = m * static_cast<uint64_t>(a->dim) * e;
        w = static_cast<uint64_t>(a->hidden) * static_cast<uint64_t>(a->dim) * e;
        out = m * static_cast<uint64_t>(a->hidden) * e;
    }
};

msel::MlpParams mlp_params(const msel_gated_mlp_args* a, void* ws) {
    msel::MlpParams p{};
    p.M = a->tokens;
    p.D = a->dim;
    p.F = a->hidden;
    p.gelu = a->activation;
    p.x = a->x;
    p.wg = a->w_gate;
    p.wu = a->w_up;
    p.ws = ws;
    return p;
}

}  // namespace

extern "C" {

msel_status msel_validate_lru_fwd(const msel_lru_args* a, const void* workspace,
                                  size_t workspace_bytes) {
    const msel_status s = check_lru(a);
    if (s != MSEL_OK) return s;
    if (a->out == nullptr) return MSEL_ERR_NULL;
    if (!aligned(a->out, 16) || !aligned(a->final_state, 4)) return MSEL_ERR_ALIGN;
    const LruBytes n(a);
    const Memory x{a->x, n.act}, ga{a->gate_a, n.act}, gx{a->gate_x, n.act}, lam{a->lam, n.lam};
    const Memory h0{a->h0, n.state}, out{a->out, n.act}, chunks{a->chunk_states, n.chunks};
    const Memory state{a->final_state, n.state};
    // final_state may be h0 itself: a row's state is read before it is written
    const Memory from = a->final_state == a->h0 ? Memory(nullptr, 0) : h0;
    if (aliased({out, chunks}, {x, ga, gx, lam, h0}) ||
        aliased({state}, {x, ga, gx, lam, from, out, chunks}))
        return MSEL_ERR_ALIAS;
    return check_workspace(workspace, workspace_bytes, lru_space(a, false).all(),
                           {x, ga, gx, lam, h0, out, state, chunks});
}

size_t msel_lru_fwd_workspace_bytes(const msel_lru_args* a) {
    return check_lru_sizes(a) == MSEL_OK ? lru_space(a, false).all() : 0;
}

msel_status msel_lru_fwd(const msel_lru_args* a, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
    const msel_status s = msel_validate_lru_fwd(a, workspace, workspace_bytes);
    if (s != MSEL_OK) return s;
    msel::LruParams p = lru_params(a);
    p.out = a->out;
    p.final_state = a->final_state;
    p.chunks = a->chunk_states;
    p.pairs = static_cast<float2*>(workspace);
    return hip_status(msel::launch_lru_fwd(p, a->dtype == MSEL_BF16, stream));
}

size_t msel_lru_bwd_workspace_bytes(const msel_lru_args* a) {
    return check_lru_sizes(a) == MSEL_OK ? lru_space(a, true).all() : 0;
}

msel_status msel_validate_lru_bwd(const msel_lru_args* a, const msel_lru_grads* g,
                                  const void* workspace, size_t workspace_bytes) {
    const msel_status s = check_lru(a);
    if (s != MSEL_OK) return s;
    if (g == nullptr || any_null({g->dout, g->dx, g->dgate_a, g->dgate_x})) return MSEL_ERR_NULL;
    if (!all_aligned({g->dout, g->dx, g->dgate_a, g->dgate_x}, 16) ||
        !all_aligned({g->dfinal_state, g->dlam, g->dh0}, 4))
        return MSEL_ERR_ALIGN;
    const LruBytes n(a);
    const Memory x{a->x, n.act}, ga{a->gate_a, n.act}, gx{a->gate_x, n.act}, lam{a->lam, n.lam};
    const Memory h0{a->h0, n.state}, chunks{a->chunk_states, n.chunks}, dout{g->dout, n.act};
    const Memory dfinal{g->dfinal_state, n.state}, dx{g->dx, n.act}, dga{g->dgate_a, n.act};
    const Memory dgx{g->dgate_x, n.act}, dlam{g->dlam, n.lam}, dh0{g->dh0, n.state};
    if (aliased({dx, dga, dgx, dlam, dh0}, {x, ga, gx, lam, h0, chunks, dout, dfinal}))
        return MSEL_ERR_ALIAS;
    return check_workspace(workspace, workspace_bytes, lru_space(a, true).all(),
                           {x, ga, gx, lam, h0, chunks, dout, dfinal, dx, dga, dgx, dlam, dh0});
}

msel_status msel_lru_bwd(const msel_lru_args* a, const msel_lru_grads* g, void* workspace,
                         size_t workspace_bytes, hipStream_t stream) {
    const msel_status s = msel_validate_lru_bwd(a, g, workspace, workspace_bytes);
    if (s != MSEL_OK) return s;
    const bool bf16 = a->dtype == MSEL_BF16;
    const LruSpace w = lru_space(a, true);
    char* const base = static_cast<char*>(workspace);
    msel::LruParams p = lru_params(a);
    p.pairs = reinterpret_cast<float2*>(base);
    p.chunks = a->chunk_states;
    if (w.chunks > 0) {
        p.chunks = reinterpret_cast<float*>(base + rounded(w.pairs));
        const msel_status t = hip_status(msel::launch_lru_fwd(p, bf16, stream));
        if (t != MSEL_OK) return t;
    }
    p.dout = g->dout;
    p.dfinal = g->dfinal_state;
    p.dx = g->dx;
    p.dga = g->dgate_a;
    p.dgx = g->dgate_x;
    p.dh0 = g->dh0;
    p.dlam = g->dlam;
    p.dlam_part = g->dlam == nullptr
                      ? nullptr
                      : reinterpret_cast<float*>(base + rounded(w.pairs) + rounded(w.chunks));
    return hip_status(msel::launch_lru_bwd(p, bf16, stream));
}

msel_status msel_validate_logprob_fwd(const msel_logprob_args* a, const void* workspace,
                                      size_t workspace_bytes) {
    const msel_status s = check_logprob(a);
    if (s != MSEL_OK) return s;
    if (a->top < 0 || a->top > a->vocab) return MSEL_ERR_SHAPE;
    if (a->top > MSEL_MAX_TOP) return MSEL_ERR_UNSUPPORTED;
    if (a->logits == nullptr || (a->logprob != nullptr && a->ids == nullptr)) return MSEL_ERR_NULL;
    if (a->top > 0 && any_null({a->top_ids, a->top_logprobs})) return MSEL_ERR_NULL;
    if (a->top == 0 && a->logprob == nullptr && a->lse == nullptr && a->entropy == nullptr)
        return MSEL_ERR_NULL;  // nothing is asked for
    if (!logprob_aligned(a)) return MSEL_ERR_ALIGN;
    const uint64_t tops = static_cast<uint64_t>(a->rows) * static_cast<uint64_t>(a->top);
    const Memory logits = logits_at(a, a->logits, a->stride), ids = ids_at(a);
    const Memory logprob = rows_at(a, a->logprob), lse = rows_at(a, a->lse);
    const Memory entropy = rows_at(a, a->entropy), top_ids{a->top_ids, tops * 8};
    const Memory top_logprobs{a->top_logprobs, tops * 4};
    if (aliased({logprob, lse, entropy, top_ids, top_logprobs}, {logits, ids}))
        return MSEL_ERR_ALIAS;
    return check_workspace(workspace, workspace_bytes, logprob_ws(a),
                           {logits, ids, logprob, lse, entropy, top_ids, top_logprobs});
}

size_t msel_logprob_fwd_workspace_bytes(const msel_logprob_args* a) {
    if (check_logprob(a) != MSEL_OK || a->top < 0 || a->top > MSEL_MAX_TOP || a->top > a->vocab)
        return 0;
    return logprob_ws(a);
}

msel_status msel_logprob_fwd(const msel_logprob_args* a, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    const msel_status s = msel_validate_logprob_fwd(a, workspace, workspace_bytes);
    if (s != MSEL_OK) return s;
    msel::LogprobParams p = logprob_params(a);
    p.top = a->top;
    p.logprob = a->logprob;
    p.lse = a->lse;
    p.entropy = a->entropy;
    p.top_ids = a->top_ids;
    p.top_logprobs = a->top_logprobs;
    p.ws = workspace;
    return hip_status(msel::launch_logprob_fwd(p, a->dtype == MSEL_BF16, stream));
}

msel_status msel_validate_logprob_bwd(const msel_logprob_args* a, const msel_logprob_grads* g) {
    const msel_status s = check_logprob(a);
    if (s != MSEL_OK) return s;
    if (g == nullptr || any_null({a->logits, a->lse, g->dlogits})) return MSEL_ERR_NULL;
    if ((g->dlogprob != nullptr && a->ids == nullptr) ||
        (g->dentropy != nullptr && a->entropy == nullptr))
        return MSEL_ERR_NULL;
    if (g->dstride < a->vocab || g->dstride > kMaxElems / a->rows) return MSEL_ERR_SHAPE;
    if (!logprob_aligned(a) || !aligned(g->dlogits, elem_bytes(a->dtype)) ||
        !all_aligned({g->dlogprob, g->dlse, g->dentropy}, 4))
        return MSEL_ERR_ALIGN;
    // in place, a row's gradient lies where the row lies; else they share nothing
    if (g->dlogits == a->logits && g->dstride != a->stride) return MSEL_ERR_SHAPE;
    const Memory dlogits = logits_at(a, g->dlogits, g->dstride);
    if (g->dlogits != a->logits && dlogits.meets(logits_at(a, a->logits, a->stride)))
        return MSEL_ERR_ALIAS;
    if (aliased({dlogits}, {ids_at(a), rows_at(a, a->lse), rows_at(a, a->entropy),
                            rows_at(a, g->dlogprob), rows_at(a, g->dlse),
                            rows_at(a, g->dentropy)}))
        return MSEL_ERR_ALIAS;
    return MSEL_OK;
}

msel_status msel_logprob_bwd(const msel_logprob_args* a, const msel_logprob_grads* g,
                             hipStream_t stream) {
    const msel_status s = msel_validate_logprob_bwd(a, g);
    if (s != MSEL_OK) return s;
    msel::LogprobParams p = logprob_params(a);
    p.in_lse = a->lse;
    p.in_entropy = a->entropy;
    p.dlogprob = g->dlogprob;
    p.dlse = g->dlse;
    p.dentropy = g->dentropy;
    p.dlogits = g->dlogits;
    p.dstride = g->dstride;
    return hip_status(msel::launch_logprob_bwd(p, a->dtype == MSEL_BF16, stream));
}

msel_status msel_validate_gated_mlp_fwd(const msel_gated_mlp_args* a, const void* workspace,
                                        size_t workspace_bytes) {
    const msel_status s = check_mlp(a);
    if (s != MSEL_OK) return s;
    if (a->out == nullptr) return MSEL_ERR_NULL;
    if (!aligned(a->out, 16)) return MSEL_ERR_ALIGN;
    const MlpBytes n(a);
    const Memory x{a->x, n.x}, wg{a->w_gate, n.w}, wu{a->w_up, n.w}, out{a->out, n.out};
    if (aliased({out}, {x, wg, wu})) return MSEL_ERR_ALIAS;
    return check_workspace(workspace, workspace_bytes, msel_gated_mlp_fwd_workspace_bytes(a),
                           {x, wg, wu, out});
}

size_t msel_gated_mlp_fwd_workspace_bytes(const msel_gated_mlp_args* a) {
    if (check_mlp_sizes(a) != MSEL_OK) return 0;
    return msel::mlp_fwd_workspace_bytes(mlp_params(a, nullptr), a->dtype == MSEL_BF16);
}

msel_status msel_gated_mlp_fwd(const msel_gated_mlp_args* a, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
    const msel_status s = msel_validate_gated_mlp_fwd(a, workspace, workspace_bytes);
    if (s != MSEL_OK) return s;
    msel::MlpParams p = mlp_params(a, workspace);
    p.out = a->out;
    return hip_status(msel::launch_mlp_fwd(p, a->dtype == MSEL_BF16, stream));
}

size_t msel_gated_mlp_bwd_workspace_bytes(const msel_gated_mlp_args* a) {
    if (check_mlp_sizes(a) != MSEL_OK) return 0;
    return msel::mlp_bwd_workspace_bytes(mlp_params(a, nullptr), a->dtype == MSEL_BF16);
}

msel_status msel_validate_gated_mlp_bwd(const msel_gated_mlp_args* a,
                                        const msel_gated_mlp_grads* g, const void* workspace,
                                        size_t workspace_bytes) {
    const msel_status s = check_mlp(a);
    if (s != MSEL_OK) return s;
    if (g == nullptr || g->dout == nullptr) return MSEL_ERR_NULL;
    if ((g->dw_gate == nullptr) != (g->dw_up == nullptr) ||
        (g->dx == nullptr && g->dw_gate == nullptr))
        return MSEL_ERR_NULL;
    if (!all_aligned({g->dout, g->dx, g->dw_gate, g->dw_up}, 16)) return MSEL_ERR_ALIGN;
    const MlpBytes n(a);
    const Memory x{a->x, n.x}, wg{a->w_gate, n.w}, wu{a->w_up, n.w}, dout{g->dout, n.out};
    const Memory dx{g->dx, n.x}, dwg{g->dw_gate, n.w}, dwu{g->dw_up, n.w};
    if (aliased({dx, dwg, dwu}, {x, wg, wu, dout})) return MSEL_ERR_ALIAS;
    return check_workspace(workspace, workspace_bytes, msel_gated_mlp_bwd_workspace_bytes(a),
                           {x, wg, wu, dout, dx, dwg, dwu});
}

msel_status msel_gated_mlp_bwd(const msel_gated_mlp_args* a, const msel_gated_mlp_grads* g,
                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const msel_status s = msel_validate_gated_mlp_bwd(a, g, workspace, workspace_bytes);
    if (s != MSEL_OK) return s;
    msel::MlpParams p = mlp_params(a, workspace);
    p.dout = g->dout;
    p.dx = g->dx;
    p.dwg = g->dw_gate;
    p.dwu = g->dw_up;
    return hip_status(msel::launch_mlp_bwd(p, a->dtype == MSEL_BF16, stream));
}

}  // extern "C"
