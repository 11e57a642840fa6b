// lm_api.cpp -- the extern "C" entry points of the operators around the scan, declared in
// include/msel.h: the norms, the embedding, the gradient norm and clipping.
//
// As in msel_api.cpp, every entry point validates its arguments on the host (no HIP call, no
// device memory touched) and only then enqueues kernels on the caller's stream; no device memory
// is allocated, and nothing is kept between calls or synchronized.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "lm_kernels.hpp"
#include "msel.h"

static_assert(MSEL_MAX_NORM_DIM == msel::kMaxNormDim, "the kernels' width limit is the boundary's");

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxRows = int64_t(1) << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool is_dtype(int32_t d) { return d == MSEL_F32 || d == MSEL_BF16; }
bool is_flag(int32_t f) { return f == 0 || f == 1; }
bool not_negative(float f) { return f >= 0.0f; }  // false for NaN
msel_status hip_status(hipError_t e) { return e == hipSuccess ? MSEL_OK : MSEL_ERR_HIP; }

template <size_t N>
bool all_aligned(const void* const (&ps)[N], uintptr_t a) {
    for (const void* p : ps)
        if (p != nullptr && !aligned(p, a)) return false;
    return true;
}

// Whether an output equals an input or another output (null ones aside).
template <size_t N, size_t M>
bool aliased(const void* const (&outs)[N], const void* const (&ins)[M]) {
    for (size_t i = 0; i < N; ++i) {
        if (outs[i] == nullptr) continue;
        for (const void* in : ins)
            if (in == outs[i]) return true;
        for (size_t j = 0; j < i; ++j)
            if (outs[j] == outs[i]) return true;
    }
    return false;
}

msel_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return MSEL_OK;
    if (ws == nullptr || have < need) return MSEL_ERR_WORKSPACE;
    return aligned(ws, 256) ? MSEL_OK : MSEL_ERR_ALIGN;
}

// ---- the norm before a block -------------------------------------------------------------

msel_status check_norm(const msel_norm_args* a) {
    if (a == nullptr) return MSEL_ERR_NULL;
    if (a->abi_version != MSEL_ABI_VERSION) return MSEL_ERR_VERSION;
    if (a->dim < 1 || a->rows < 1 || a->rows > kMaxElems / a->dim)
        return MSEL_ERR_SHAPE;
    if (!is_dtype(a->dtype) || !is_dtype(a->residual_dtype)) return MSEL_ERR_DTYPE;
    if (a->residual_dtype != a->dtype && a->residual_dtype != MSEL_F32) return MSEL_ERR_DTYPE;
    if (a->dim > MSEL_MAX_NORM_DIM) return MSEL_ERR_UNSUPPORTED;
    if (!not_negative(a->eps)) return MSEL_ERR_SHAPE;
    if (a->weight != nullptr && !aligned(a->weight, 4)) return MSEL_ERR_ALIGN;
    return MSEL_OK;
}

msel::RowNormParams norm_params(const msel_norm_args* a) {
    msel::RowNormParams p{};
    p.rows = a->rows;
    p.groups = 1;
    p.n = a->dim;
    p.scale = a->scale;
    p.eps = a->eps;
    p.w = a->weight;
    return p;
}

size_t norm_ws(const msel_norm_args* a) {
    return static_cast<size_t>(msel::row_norm_partials(
               a->rows, 1, a->dim, msel::NormMode::kResidual, a->dtype == MSEL_BF16,
               a->residual_dtype == MSEL_BF16)) *
           static_cast<size_t>(a->dim) * sizeof(float);
}

// ---- the gated norm ----------------------------------------------------------------------

msel_status check_gated(const msel_gated_norm_args* a) {
    if (a == nullptr) return MSEL_ERR_NULL;
    if (a->abi_version != MSEL_ABI_VERSION) return MSEL_ERR_VERSION;
    if (a->batch < 1 || a->dim < 1 || a->seqlen < 1 || a->groups < 1) return MSEL_ERR_SHAPE;
    if (static_cast<int64_t>(a->batch) * a->dim > kMaxRows || a->seqlen > MSEL_MAX_SEQLEN ||
        static_cast<int64_t>(a->batch) * a->seqlen > kMaxRows ||
        static_cast<int64_t>(a->batch) * a->seqlen * a->dim > kMaxElems ||
        a->dim % a->groups != 0)
        return MSEL_ERR_SHAPE;
    if (!is_dtype(a->dtype) || !is_flag(a->gate_first)) return MSEL_ERR_DTYPE;
    if (!is_flag(a->layout) || !is_flag(a->out_layout)) return MSEL_ERR_DTYPE;
    if (!not_negative(a->eps)) return MSEL_ERR_SHAPE;
    if (a->dim / a->groups > MSEL_MAX_NORM_DIM || a->groups > MSEL_MAX_NORM_GROUPS ||
        (a->layout == MSEL_BLD && a->out_layout == MSEL_BDL))
        return MSEL_ERR_UNSUPPORTED;
    if (a->x == nullptr || a->z == nullptr) return MSEL_ERR_NULL;
    if (!aligned(a->x, 16) || !aligned(a->z, 16)) return MSEL_ERR_ALIGN;
    if (a->weight != nullptr && !aligned(a->weight, 4)) return MSEL_ERR_ALIGN;
    return MSEL_OK;
}

// Rows of contiguous channels: [batch, seqlen, dim], or one step, where the layouts agree.
bool gated_by_rows(const msel_gated_norm_args* a) {
    return a->layout == MSEL_BLD || a->seqlen == 1;
}

msel::NormMode gated_mode(const msel_gated_norm_args* a) {
    return a->gate_first ? msel::NormMode::kGateFirst : msel::NormMode::kGateLast;
}

msel::RowNormParams gated_rows(const msel_gated_norm_args* a) {
    msel::RowNormParams p{};
    p.rows = static_cast<int64_t>(a->batch) * a->seqlen;
    p.groups = a->groups;
    p.n = a->dim / a->groups;
    p.scale = 1.0f;
    p.eps = a->eps;
    p.a = a->x;
    p.b = a->z;
    p.w = a->weight;
    return p;
}

msel::TileNormParams gated_tiles(const msel_gated_norm_args* a) {
    msel::TileNormParams p{};
    p.B = a->batch;
    p.D = a->dim;
    p.L = a->seqlen;
    p.groups = a->groups;
    p.n = a->dim / a->groups;
    p.eps = a->eps;
    p.out_bld = a->out_layout == MSEL_BLD ? 1 : 0;
    p.x = a->x;
    p.z = a->z;
    p.w = a->weight;
    return p;
}

size_t gated_ws(const msel_gated_norm_args* a) {
    const bool bf16 = a->dtype == MSEL_BF16;
    const int64_t parts =
        gated_by_rows(a)
            ? msel::row_norm_partials(static_cast<int64_t>(a->batch) * a->seqlen, a->groups,
                                      a->dim / a->groups, gated_mode(a), bf16, bf16)
            : msel::tile_norm_partials(a->batch, a->groups, a->dim / a->groups, a->seqlen, bf16);
    return static_cast<size_t>(parts) * static_cast<size_t>(a->dim) * sizeof(float);
}

// ---- the embedding -----------------------------------------------------------------------

msel_status check_embed(const msel_embed_args* a) {
    if (a == nullptr) return MSEL_ERR_NULL;
    if (a->abi_version != MSEL_ABI_VERSION || a->reserved != 0) return MSEL_ERR_VERSION;
    if (a->vocab < 1 || a->dim < 1 || a->tokens < 1 || a->vocab > kMaxRows ||
        a->tokens > kMaxRows || static_cast<int64_t>(a->vocab) * a->dim > kMaxElems ||
        a->tokens * a->dim > kMaxElems)
        return MSEL_ERR_SHAPE;
    if (!is_dtype(a->dtype) || !is_flag(a->ids_64bit)) return MSEL_ERR_DTYPE;
    if (a->dim > MSEL_MAX_NORM_DIM) return MSEL_ERR_UNSUPPORTED;
    if (a->ids == nullptr) return MSEL_ERR_NULL;
    return aligned(a->ids, a->ids_64bit ? 8 : 4) ? MSEL_OK : MSEL_ERR_ALIGN;
}

msel::EmbedParams embed_params(const msel_embed_args* a) {
    msel::EmbedParams p{};
    p.tokens = a->tokens;
    p.vocab = a->vocab;
    p.dim = a->dim;
    p.ids64 = a->ids_64bit;
    p.padding_idx = a->padding_idx;
    p.scale = a->scale;
    p.ids = a->ids;
    return p;
}

// ---- gradient norm and clipping ----------------------------------------------------------

msel::GradTensor read_tensor(const void* list, const void* outs, int i) {
    const msel_tensor& t = static_cast<const msel_tensor*>(list)[i];
    void* dst = outs != nullptr ? static_cast<const msel_tensor*>(outs)[i].data : nullptr;
    return msel::GradTensor{t.data, dst, t.numel, t.dtype == MSEL_BF16};
}

msel_status check_tensor(const msel_tensor& t) {
    if (t.numel < 0 || t.numel > kMaxElems) return MSEL_ERR_SHAPE;
    if (!is_dtype(t.dtype)) return MSEL_ERR_DTYPE;
    if (t.reserved != 0) return MSEL_ERR_VERSION;
    if (t.numel == 0) return MSEL_OK;
    if (t.data == nullptr) return MSEL_ERR_NULL;
    return aligned(t.data, t.dtype == MSEL_BF16 ? 2 : 4) ? MSEL_OK : MSEL_ERR_ALIGN;
}

msel_status check_grads(const msel_grad_args* a) {
    if (a == nullptr) return MSEL_ERR_NULL;
    if (a->abi_version != MSEL_ABI_VERSION) return MSEL_ERR_VERSION;
    if (a->count < 0 || a->count > MSEL_MAX_GRAD_TENSORS) return MSEL_ERR_SHAPE;
    if (a->count > 0 && a->tensors == nullptr) return MSEL_ERR_NULL;
    int64_t total = 0;
    for (int32_t i = 0; i < a->count; ++i) {
        const msel_status s = check_tensor(a->tensors[i]);
        if (s != MSEL_OK) return s;
        total += a->tensors[i].numel;
        if (total > kMaxElems) return MSEL_ERR_SHAPE;
    }
    return MSEL_OK;
}

// A stretch of memory; ranges by their addresses.
struct Range {
    uintptr_t begin, end;
    bool operator<(const Range& o) const { return begin < o.begin; }
    bool meets(const Range& o) const { return begin < o.end && o.begin < end; }
};
constexpr size_t kStackRanges = 1024;  // longer lists take the host's heap

// Whether something that clipping writes (a destination, norm, the workspace) shares memory with
// anything else that it reads or writes; a destination may be its own entry's source.  The blocks
// of a launch scale their chunks in no order, so such calls would have no one result.  whole: the
// ranges are the tensors' bytes; else their first ones, which finds equal addresses alone.
// In the order of addresses, a range meets an earlier one if it begins below the largest end so
// far.  Lists are mostly in that order already, and are sorted only where they are not.
msel_status check_overlap(const msel_grad_args* a, const void* ws, size_t ws_bytes, bool whole) {
    Range stack[kStackRanges];
    const size_t most = 2 * static_cast<size_t>(a->count);
    Range* const heap = most > kStackRanges ? new (std::nothrow) Range[most] : nullptr;
    if (most > kStackRanges && heap == nullptr) return MSEL_ERR_TOO_LARGE;
    const auto range = [&](const void* p, size_t bytes) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        return Range{at, at + (whole ? bytes : 1)};
    };
    // destinations from the front, the sources that are none from the middle
    Range* const dst = heap != nullptr ? heap : stack;
    Range* const src = dst + a->count;
    size_t nd = 0, ns = 0;
    for (int32_t i = 0; i < a->count; ++i) {
        const msel_tensor& t = a->tensors[i];
        if (t.numel == 0) continue;
        const size_t bytes = static_cast<size_t>(t.numel) * (t.dtype == MSEL_BF16 ? 2 : 4);
        dst[nd++] = range(a->outs[i].data, bytes);
        if (t.data != a->outs[i].data) src[ns++] = range(t.data, bytes);
    }
    if (!std::is_sorted(dst, dst + nd)) std::sort(dst, dst + nd);
    if (!std::is_sorted(src, src + ns)) std::sort(src, src + ns);
    const Range norm = range(a->norm, sizeof(float)), work = range(ws, ws_bytes);
    bool meet = norm.meets(work);
    uintptr_t any = 0, written = 0;  // the largest ends so far
    for (size_t i = 0, j = 0; (i < nd || j < ns) && !meet;) {
        const bool out = j == ns || (i < nd && dst[i] < src[j]);
        const Range& r = out ? dst[i++] : src[j++];
        meet = r.begin < (out ? any : written) || r.meets(norm) || r.meets(work);
        any = std::max(any, r.end);
        if (out) written = std::max(written, r.end);
    }
    delete[] heap;
    return meet ? MSEL_ERR_ALIAS : MSEL_OK;
}

msel::GradNormParams grad_params(const msel_grad_args* a, void* ws) {
    msel::GradNormParams p{};
    p.count = a->count;
    p.list = a->tensors;
    p.outs = a->outs;
    p.read = read_tensor;
    p.max_norm = a->max_norm;
    p.eps = a->eps;
    p.norm = a->norm;
    p.partials = static_cast<double*>(ws);
    return p;
}

size_t grad_ws(const msel_grad_args* a) {
    // one more for the scaling factor
    return static_cast<size_t>(msel::grad_partials(grad_params(a, nullptr)) + 1) * sizeof(double);
}

msel_status check_norm_call(const msel_grad_args* a, const void* ws, size_t ws_bytes, size_t& need) {
    const msel_status s = check_grads(a);
    if (s != MSEL_OK) return s;
    if (a->norm == nullptr) return MSEL_ERR_NULL;
    if (!aligned(a->norm, 4)) return MSEL_ERR_ALIGN;
    for (int32_t i = 0; i < a->count; ++i)
        if (a->tensors[i].numel > 0 &&
            (a->tensors[i].data == a->norm || a->tensors[i].data == ws))
            return MSEL_ERR_ALIAS;
    need = grad_ws(a);
    return check_workspace(ws, ws_bytes, need);
}

msel_status check_clip_call(const msel_grad_args* a, const void* ws, size_t ws_bytes, bool whole) {
    size_t need = 0;
    const msel_status s = check_norm_call(a, ws, ws_bytes, need);
    if (s != MSEL_OK) return s;
    if (!not_negative(a->max_norm) || !not_negative(a->eps)) return MSEL_ERR_SHAPE;
    if (a->count > 0 && a->outs == nullptr) return MSEL_ERR_NULL;
    for (int32_t i = 0; i < a->count; ++i) {
        const msel_status t = check_tensor(a->outs[i]);
        if (t != MSEL_OK) return t;
        if (a->outs[i].numel != a->tensors[i].numel) return MSEL_ERR_SHAPE;
        if (a->outs[i].dtype != a->tensors[i].dtype) return MSEL_ERR_DTYPE;
    }
    return check_overlap(a, ws, need, whole);
}

}  // namespace

extern "C" {

msel_status msel_validate_norm_fwd(const msel_norm_args* a) {
    const msel_status s = check_norm(a);
    if (s != MSEL_OK) return s;
    if (a->x == nullptr || a->out == nullptr) return MSEL_ERR_NULL;
    const void* const act[] = {a->x, a->residual, a->out, a->residual_out};
    if (!all_aligned(act, 16)) return MSEL_ERR_ALIGN;
    const void* const outs[] = {a->out};
    const void* const ins[] = {a->x, a->residual, a->weight, a->residual_out};
    // residual_out may be residual itself: each row is read before it is written
    const void* const rest[] = {a->residual_out == a->residual ? nullptr : a->residual_out};
    if (aliased(outs, ins) || aliased(rest, {a->x, a->residual, static_cast<const void*>(a->weight)}))
        return MSEL_ERR_ALIAS;
    return a->residual_out != nullptr && a->residual_out == a->weight ? MSEL_ERR_ALIAS : MSEL_OK;
}

size_t msel_norm_bwd_workspace_bytes(const msel_norm_args* a) {
    return check_norm(a) == MSEL_OK ? norm_ws(a) : 0;
}

msel_status msel_validate_norm_bwd(const msel_norm_args* a, const msel_norm_grads* g,
                                   const void* workspace, size_t workspace_bytes) {
    msel_status s = check_norm(a);
    if (s != MSEL_OK) return s;
    if (g == nullptr || g->s == nullptr || g->dout == nullptr) return MSEL_ERR_NULL;
    if (g->dx == nullptr && g->dresidual == nullptr && g->dweight == nullptr) return MSEL_ERR_NULL;
    const void* const act[] = {g->s, g->dout, g->dresidual_out, g->dx, g->dresidual};
    if (!all_aligned(act, 16)) return MSEL_ERR_ALIGN;
    if (g->dweight != nullptr && !aligned(g->dweight, 4)) return MSEL_ERR_ALIGN;
    const void* const outs[] = {g->dx, g->dweight, g->dresidual};
    // dresidual may be dresidual_out itself: each row is read before it is written
    const void* const ins[] = {g->s, g->dout, a->weight,
                               g->dresidual == g->dresidual_out ? nullptr : g->dresidual_out};
    if (aliased(outs, ins)) return MSEL_ERR_ALIAS;
    s = check_workspace(workspace, workspace_bytes, g->dweight != nullptr ? norm_ws(a) : 0);
    if (s != MSEL_OK) return s;
    const void* const ws[] = {g->dweight != nullptr ? workspace : nullptr};
    return aliased(ws, {g->s, g->dout, g->dresidual_out, static_cast<const void*>(a->weight), g->dx,
                        g->dresidual, static_cast<const void*>(g->dweight)})
               ? MSEL_ERR_ALIAS
               : MSEL_OK;
}

msel_status msel_norm_fwd(const msel_norm_args* a, hipStream_t stream) {
    const msel_status s = msel_validate_norm_fwd(a);
    if (s != MSEL_OK) return s;
    msel::RowNormParams p = norm_params(a);
    p.a = a->x;
    p.b = a->residual;
    p.out = a->out;
    p.out2 = a->residual_out;
    return hip_status(msel::launch_row_norm_fwd(p, msel::NormMode::kResidual,
                                                a->dtype == MSEL_BF16,
                                                a->residual_dtype == MSEL_BF16, stream));
}

msel_status msel_norm_bwd(const msel_norm_args* a, const msel_norm_grads* g, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
    const msel_status s = msel_validate_norm_bwd(a, g, workspace, workspace_bytes);
    if (s != MSEL_OK) return s;
    msel::RowNormParams p = norm_params(a);
    p.a = g->s;
    p.b = g->dresidual_out;
    p.dout = g->dout;
    p.out = g->dx;
    p.out2 = g->dresidual;
    p.dw = g->dweight;
    p.dw_part = g->dweight != nullptr ? static_cast<float*>(workspace) : nullptr;
    return hip_status(msel::launch_row_norm_bwd(p, msel::NormMode::kResidual,
                                                a->dtype == MSEL_BF16,
                                                a->residual_dtype == MSEL_BF16, stream));
}

msel_status msel_validate_gated_norm_fwd(const msel_gated_norm_args* a) {
    const msel_status s = check_gated(a);
    if (s != MSEL_OK) return s;
    if (a->out == nullptr) return MSEL_ERR_NULL;
    if (!aligned(a->out, 16)) return MSEL_ERR_ALIGN;
    const void* const outs[] = {a->out};
    return aliased(outs, {a->x, a->z, static_cast<const void*>(a->weight)}) ? MSEL_ERR_ALIAS
                                                                            : MSEL_OK;
}

size_t msel_gated_norm_bwd_workspace_bytes(const msel_gated_norm_args* a) {
    return check_gated(a) == MSEL_OK ? gated_ws(a) : 0;
}

msel_status msel_validate_gated_norm_bwd(const msel_gated_norm_args* a,
                                         const msel_gated_norm_grads* g, const void* workspace,
                                         size_t workspace_bytes) {
    msel_status s = check_gated(a);
    if (s != MSEL_OK) return s;
    if (g == nullptr || g->dout == nullptr || g->dx == nullptr || g->dz == nullptr)
        return MSEL_ERR_NULL;
    const void* const act[] = {g->dout, g->dx, g->dz};
    if (!all_aligned(act, 16)) return MSEL_ERR_ALIGN;
    if (g->dweight != nullptr && !aligned(g->dweight, 4)) return MSEL_ERR_ALIGN;
    const void* const outs[] = {g->dx, g->dz, g->dweight};
    if (aliased(outs, {a->x, a->z, static_cast<const void*>(a->weight), g->dout}))
        return MSEL_ERR_ALIAS;
    s = check_workspace(workspace, workspace_bytes, g->dweight != nullptr ? gated_ws(a) : 0);
    if (s != MSEL_OK) return s;
    const void* const ws[] = {g->dweight != nullptr ? workspace : nullptr};
    return aliased(ws, {a->x, a->z, static_cast<const void*>(a->weight), g->dout, g->dx, g->dz,
                        static_cast<const void*>(g->dweight)})
               ? MSEL_ERR_ALIAS
               : MSEL_OK;
}

msel_status msel_gated_norm_fwd(const msel_gated_norm_args* a, hipStream_t stream) {
    const msel_status s = msel_validate_gated_norm_fwd(a);
    if (s != MSEL_OK) return s;
    const bool bf16 = a->dtype == MSEL_BF16;
    if (gated_by_rows(a)) {
        msel::RowNormParams p = gated_rows(a);
        p.out = a->out;
        return hip_status(msel::launch_row_norm_fwd(p, gated_mode(a), bf16, bf16, stream));
    }
    msel::TileNormParams p = gated_tiles(a);
    p.out = a->out;
    return hip_status(msel::launch_tile_norm_fwd(p, a->gate_first != 0, bf16, stream));
}

msel_status msel_gated_norm_bwd(const msel_gated_norm_args* a, const msel_gated_norm_grads* g,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const msel_status s = msel_validate_gated_norm_bwd(a, g, workspace, workspace_bytes);
    if (s != MSEL_OK) return s;
    const bool bf16 = a->dtype == MSEL_BF16;
    float* part = g->dweight != nullptr ? static_cast<float*>(workspace) : nullptr;
    if (gated_by_rows(a)) {
        msel::RowNormParams p = gated_rows(a);
        p.dout = g->dout;
        p.out = g->dx;
        p.out2 = g->dz;
        p.dw_part = part;
        p.dw = g->dweight;
        return hip_status(msel::launch_row_norm_bwd(p, gated_mode(a), bf16, bf16, stream));
    }
    msel::TileNormParams p = gated_tiles(a);
    p.dout = g->dout;
    p.out = g->dx;
    p.dz = g->dz;
    p.dw_part = part;
    p.dw = g->dweight;
    return hip_status(msel::launch_tile_norm_bwd(p, a->gate_first != 0, bf16, stream));
}

msel_status msel_validate_embed_fwd(const msel_embed_args* a) {
    const msel_status s = check_embed(a);
    if (s != MSEL_OK) return s;
    if (!is_dtype(a->weight_dtype)) return MSEL_ERR_DTYPE;
    if (a->weight == nullptr || a->out == nullptr) return MSEL_ERR_NULL;
    if (!aligned(a->weight, 16) || !aligned(a->out, 16)) return MSEL_ERR_ALIGN;
    const void* const outs[] = {a->out};
    return aliased(outs, {a->ids, a->weight}) ? MSEL_ERR_ALIAS : MSEL_OK;
}

size_t msel_embed_bwd_workspace_bytes(const msel_embed_args* a) {
    return check_embed(a) == MSEL_OK ? msel::embed_workspace_bytes(a->tokens, a->vocab, a->dim) : 0;
}

msel_status msel_validate_embed_bwd(const msel_embed_args* a, const msel_embed_grads* g,
                                    const void* workspace, size_t workspace_bytes) {
    msel_status s = check_embed(a);
    if (s != MSEL_OK) return s;
    if (g == nullptr || g->dout == nullptr || g->dweight == nullptr) return MSEL_ERR_NULL;
    const void* const act[] = {g->dout, g->base, g->dweight};
    if (!all_aligned(act, 16)) return MSEL_ERR_ALIGN;
    const void* const outs[] = {g->dweight};
    if (aliased(outs, {a->ids, g->dout})) return MSEL_ERR_ALIAS;
    s = check_workspace(workspace, workspace_bytes, msel_embed_bwd_workspace_bytes(a));
    if (s != MSEL_OK) return s;
    const void* const ws[] = {workspace};
    return aliased(ws, {a->ids, g->dout, static_cast<const void*>(g->base),
                        static_cast<const void*>(g->dweight)})
               ? MSEL_ERR_ALIAS
               : MSEL_OK;
}

msel_status msel_embed_fwd(const msel_embed_args* a, hipStream_t stream) {
    const msel_status s = msel_validate_embed_fwd(a);
    if (s != MSEL_OK) return s;
    msel::EmbedParams p = embed_params(a);
    p.w = a->weight;
    p.out = a->out;
    return hip_status(msel::launch_embed_fwd(p, a->weight_dtype == MSEL_BF16,
                                             a->dtype == MSEL_BF16, stream));
}

msel_status msel_embed_bwd(const msel_embed_args* a, const msel_embed_grads* g, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
    const msel_status s = msel_validate_embed_bwd(a, g, workspace, workspace_bytes);
    if (s != MSEL_OK) return s;
    msel::EmbedParams p = embed_params(a);
    p.dout = g->dout;
    p.base = g->base;
    p.dw = g->dweight;
    p.ws = workspace;
    return hip_status(msel::launch_embed_bwd(p, a->dtype == MSEL_BF16, stream));
}

size_t msel_grad_workspace_bytes(const msel_grad_args* a) {
    return check_grads(a) == MSEL_OK ? grad_ws(a) : 0;
}

msel_status msel_validate_grad_norm(const msel_grad_args* a, const void* workspace,
                                    size_t workspace_bytes) {
    size_t need = 0;
    return check_norm_call(a, workspace, workspace_bytes, need);
}

msel_status msel_validate_grad_clip(const msel_grad_args* a, const void* workspace,
                                    size_t workspace_bytes) {
    return check_clip_call(a, workspace, workspace_bytes, false);
}

msel_status msel_grad_norm(const msel_grad_args* a, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
    const msel_status s = msel_validate_grad_norm(a, workspace, workspace_bytes);
    if (s != MSEL_OK) return s;
    msel::GradNormParams p = grad_params(a, workspace);
    p.outs = nullptr;
    p.max_norm = INFINITY;
    p.eps = 0.0f;
    return hip_status(msel::launch_grad_norm(p, false, stream));
}

msel_status msel_grad_clip(const msel_grad_args* a, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
    const msel_status s = check_clip_call(a, workspace, workspace_bytes, true);
    if (s != MSEL_OK) return s;
    return hip_status(msel::launch_grad_norm(grad_params(a, workspace), true, stream));
}

}  // extern "C"
