/*
 * Host-side code of the operators around the scan (norms, embedding, gradient clipping) under
 * AddressSanitizer and UndefinedBehaviorSanitizer.
 *
 * Built by tests/test_lm_sanitizers.py against a build of the library's sources with the
 * sanitizers on the host side: every check is run on valid arguments and on each kind of invalid
 * one, workspaces are sized from the smallest to the largest sizes, and the entry points are
 * called with invalid arguments, on which they return before any HIP call.  Device pointers are
 * fake addresses that nothing dereferences.  Exit status 0 when every expectation holds.
 */
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "msel.h"

static int failures = 0;
static uintptr_t next_addr = 0x10000000u;

static void *fake(void) {
    void *p = (void *)next_addr;
    next_addr += 0x100000u;
    return p;
}

#define EXPECT(expr, want)                                                               \
    do {                                                                                 \
        long long got_ = (long long)(expr);                                              \
        if (got_ != (long long)(want)) {                                                 \
            fprintf(stderr, "%s:%d: %s = %lld, expected %lld\n", __FILE__, __LINE__,      \
                    #expr, got_, (long long)(want));                                     \
            ++failures;                                                                  \
        }                                                                                \
    } while (0)

/* one field of a copy changed, then the check */
#define WITH(type, from, field, value, call, want) \
    do {                                           \
        type x = from;                             \
        x.field = value;                           \
        EXPECT(call, want);                        \
    } while (0)

static const float bad_floats[] = {-1.0f, NAN};

static void norm(void) {
    msel_norm_args a;
    memset(&a, 0, sizeof a);
    a.abi_version = MSEL_ABI_VERSION;
    a.dim = 768;
    a.rows = 100;
    a.dtype = MSEL_BF16;
    a.residual_dtype = MSEL_F32;
    a.scale = 1.0f;
    a.eps = 1e-5f;
    a.x = fake();
    a.residual = fake();
    a.weight = fake();
    a.out = fake();
    a.residual_out = (void *)a.residual;
    EXPECT(msel_validate_norm_fwd(&a), MSEL_OK);
    EXPECT(msel_validate_norm_fwd(NULL), MSEL_ERR_NULL);
    EXPECT(msel_norm_fwd(NULL, NULL), MSEL_ERR_NULL);
#define N(field, value, want) WITH(msel_norm_args, a, field, value, msel_norm_fwd(&x, NULL), want)
    N(abi_version, -1, MSEL_ERR_VERSION);
    N(dim, 0, MSEL_ERR_SHAPE);
    N(dim, INT32_MIN, MSEL_ERR_SHAPE);
    N(dim, MSEL_MAX_NORM_DIM + 1, MSEL_ERR_UNSUPPORTED);
    N(dim, INT32_MAX, MSEL_ERR_UNSUPPORTED);
    N(rows, 0, MSEL_ERR_SHAPE);
    N(rows, INT64_MIN, MSEL_ERR_SHAPE);
    N(rows, INT64_MAX, MSEL_ERR_SHAPE);
    N(rows, (int64_t)1 << 40, MSEL_ERR_SHAPE);
    WITH(msel_norm_args, a, rows, (int64_t)1 << 40,
         (x.dim = INT32_MAX, msel_norm_fwd(&x, NULL)), MSEL_ERR_SHAPE);
    N(dtype, 2, MSEL_ERR_DTYPE);
    N(residual_dtype, -1, MSEL_ERR_DTYPE);
    for (int i = 0; i < 2; ++i) N(eps, bad_floats[i], MSEL_ERR_SHAPE);
    N(x, NULL, MSEL_ERR_NULL);
    N(out, NULL, MSEL_ERR_NULL);
    N(x, (char *)a.x + 2, MSEL_ERR_ALIGN);
    N(weight, (float *)((char *)a.weight + 2), MSEL_ERR_ALIGN);
    N(out, (void *)a.x, MSEL_ERR_ALIAS);
    N(residual_out, (void *)a.x, MSEL_ERR_ALIAS);
    N(residual_out, (void *)a.weight, MSEL_ERR_ALIAS);
    msel_norm_grads g;
    memset(&g, 0, sizeof g);
    g.s = fake();
    g.dout = fake();
    g.dx = fake();
    g.dresidual_out = fake();
    g.dresidual = (void *)g.dresidual_out;
    g.dweight = fake();
    void *ws = fake();
    const size_t need = msel_norm_bwd_workspace_bytes(&a);
    EXPECT(need > 0, 1);
    EXPECT(msel_norm_bwd_workspace_bytes(NULL), 0);
    EXPECT(msel_validate_norm_bwd(&a, &g, ws, need), MSEL_OK);
    EXPECT(msel_norm_bwd(&a, &g, ws, need - 1, NULL), MSEL_ERR_WORKSPACE);
    EXPECT(msel_norm_bwd(&a, &g, NULL, need, NULL), MSEL_ERR_WORKSPACE);
    EXPECT(msel_norm_bwd(&a, &g, (char *)ws + 16, need, NULL), MSEL_ERR_ALIGN);
    EXPECT(msel_norm_bwd(&a, &g, g.dx, need, NULL), MSEL_ERR_ALIAS);
    EXPECT(msel_norm_bwd(&a, NULL, ws, need, NULL), MSEL_ERR_NULL);
#define G(field, value, want) \
    WITH(msel_norm_grads, g, field, value, msel_validate_norm_bwd(&a, &x, ws, need), want)
    G(s, NULL, MSEL_ERR_NULL);
    G(dout, NULL, MSEL_ERR_NULL);
    G(dx, (void *)g.dout, MSEL_ERR_ALIAS);
    G(dweight, (float *)g.dx, MSEL_ERR_ALIAS);
    G(dweight, NULL, MSEL_OK);
    G(dx, (char *)g.dx + 8, MSEL_ERR_ALIGN);
    /* every size up to the limits gives a workspace, and no overflow on the way */
    for (int32_t d = 1; d <= MSEL_MAX_NORM_DIM; d += 1 + d / 3)
        for (int64_t r = 1; r * d <= (int64_t)1 << 40; r = r * 7 + 1)
            WITH(msel_norm_args, a, dim, d, (x.rows = r, msel_norm_bwd_workspace_bytes(&x) > 0), 1);
#undef N
#undef G
}

static void gated(void) {
    msel_gated_norm_args a;
    memset(&a, 0, sizeof a);
    a.abi_version = MSEL_ABI_VERSION;
    a.batch = 2;
    a.dim = 96;
    a.seqlen = 50;
    a.groups = 4;
    a.dtype = MSEL_BF16;
    a.layout = MSEL_BDL;
    a.out_layout = MSEL_BLD;
    a.gate_first = 1;
    a.eps = 1e-5f;
    a.x = fake();
    a.z = fake();
    a.weight = fake();
    a.out = fake();
    EXPECT(msel_validate_gated_norm_fwd(&a), MSEL_OK);
    EXPECT(msel_gated_norm_fwd(NULL, NULL), MSEL_ERR_NULL);
#define N(field, value, want) \
    WITH(msel_gated_norm_args, a, field, value, msel_gated_norm_fwd(&x, NULL), want)
    N(abi_version, 0, MSEL_ERR_VERSION);
    N(batch, 0, MSEL_ERR_SHAPE);
    N(batch, INT32_MAX, MSEL_ERR_SHAPE);
    N(dim, -96, MSEL_ERR_SHAPE);
    N(dim, 97, MSEL_ERR_SHAPE);
    N(dim, INT32_MAX, MSEL_ERR_SHAPE);
    N(seqlen, 0, MSEL_ERR_SHAPE);
    N(seqlen, INT32_MAX, MSEL_ERR_SHAPE);
    N(groups, 0, MSEL_ERR_SHAPE);
    N(groups, 5, MSEL_ERR_SHAPE);
    N(dtype, 7, MSEL_ERR_DTYPE);
    N(gate_first, 2, MSEL_ERR_DTYPE);
    N(layout, -1, MSEL_ERR_DTYPE);
    N(out_layout, 2, MSEL_ERR_DTYPE);
    N(eps, NAN, MSEL_ERR_SHAPE);
    N(x, NULL, MSEL_ERR_NULL);
    N(z, NULL, MSEL_ERR_NULL);
    N(out, NULL, MSEL_ERR_NULL);
    N(z, (char *)a.z + 4, MSEL_ERR_ALIGN);
    N(out, (void *)a.z, MSEL_ERR_ALIAS);
    N(dim, 4 * (MSEL_MAX_NORM_DIM + 1), MSEL_ERR_UNSUPPORTED);
    WITH(msel_gated_norm_args, a, layout, MSEL_BLD,
         (x.out_layout = MSEL_BDL, msel_gated_norm_fwd(&x, NULL)), MSEL_ERR_UNSUPPORTED);
    WITH(msel_gated_norm_args, a, groups, MSEL_MAX_NORM_GROUPS + 1,
         (x.dim = x.groups, msel_gated_norm_fwd(&x, NULL)), MSEL_ERR_UNSUPPORTED);
    msel_gated_norm_grads g;
    memset(&g, 0, sizeof g);
    g.dout = fake();
    g.dx = fake();
    g.dz = fake();
    g.dweight = fake();
    void *ws = fake();
    const size_t need = msel_gated_norm_bwd_workspace_bytes(&a);
    EXPECT(need > 0, 1);
    EXPECT(msel_validate_gated_norm_bwd(&a, &g, ws, need), MSEL_OK);
    EXPECT(msel_gated_norm_bwd(&a, &g, ws, 0, NULL), MSEL_ERR_WORKSPACE);
    EXPECT(msel_gated_norm_bwd(&a, NULL, ws, need, NULL), MSEL_ERR_NULL);
#define G(field, value, want) \
    WITH(msel_gated_norm_grads, g, field, value, msel_validate_gated_norm_bwd(&a, &x, ws, need), want)
    G(dx, NULL, MSEL_ERR_NULL);
    G(dz, NULL, MSEL_ERR_NULL);
    G(dout, NULL, MSEL_ERR_NULL);
    G(dz, g.dx, MSEL_ERR_ALIAS);
    G(dx, (void *)a.x, MSEL_ERR_ALIAS);
    G(dweight, (float *)ws, MSEL_ERR_ALIAS);
    for (int32_t l = 0; l < 2; ++l)
        for (int32_t L = 1; L <= 1 << 28; L = L * 5 + 2)
            for (int32_t b = 1; (int64_t)b * L <= 1 << 30 && b <= 1 << 23; b = b * 9 + 1)
                WITH(msel_gated_norm_args, a, layout, l,
                     (x.out_layout = MSEL_BLD, x.seqlen = L, x.batch = b,
                      msel_gated_norm_bwd_workspace_bytes(&x) > 0), 1);
#undef N
#undef G
}

static void embed(void) {
    msel_embed_args a;
    memset(&a, 0, sizeof a);
    a.abi_version = MSEL_ABI_VERSION;
    a.vocab = 1000;
    a.dim = 64;
    a.ids_64bit = 1;
    a.tokens = 500;
    a.padding_idx = -1;
    a.scale = 1.0f;
    a.ids = fake();
    a.weight = fake();
    a.out = fake();
    EXPECT(msel_validate_embed_fwd(&a), MSEL_OK);
    EXPECT(msel_embed_fwd(NULL, NULL), MSEL_ERR_NULL);
#define N(field, value, want) WITH(msel_embed_args, a, field, value, msel_embed_fwd(&x, NULL), want)
    N(abi_version, 99, MSEL_ERR_VERSION);
    N(reserved, 1, MSEL_ERR_VERSION);
    N(vocab, 0, MSEL_ERR_SHAPE);
    N(vocab, INT32_MAX, MSEL_ERR_SHAPE);
    N(dim, 0, MSEL_ERR_SHAPE);
    N(dim, MSEL_MAX_NORM_DIM + 1, MSEL_ERR_UNSUPPORTED);
    N(tokens, 0, MSEL_ERR_SHAPE);
    N(tokens, INT64_MAX, MSEL_ERR_SHAPE);
    N(ids_64bit, 3, MSEL_ERR_DTYPE);
    N(dtype, 5, MSEL_ERR_DTYPE);
    N(weight_dtype, 5, MSEL_ERR_DTYPE);
    N(ids, NULL, MSEL_ERR_NULL);
    N(ids, (char *)a.ids + 4, MSEL_ERR_ALIGN);
    N(weight, NULL, MSEL_ERR_NULL);
    N(out, (void *)a.weight, MSEL_ERR_ALIAS);
    msel_embed_grads g;
    memset(&g, 0, sizeof g);
    g.dout = fake();
    g.dweight = fake();
    g.base = g.dweight;
    void *ws = fake();
    const size_t need = msel_embed_bwd_workspace_bytes(&a);
    EXPECT(need > 0, 1);
    EXPECT(msel_embed_bwd_workspace_bytes(NULL), 0);
    EXPECT(msel_validate_embed_bwd(&a, &g, ws, need), MSEL_OK);
    EXPECT(msel_embed_bwd(&a, &g, ws, need - 1, NULL), MSEL_ERR_WORKSPACE);
    EXPECT(msel_embed_bwd(&a, NULL, ws, need, NULL), MSEL_ERR_NULL);
#define G(field, value, want) \
    WITH(msel_embed_grads, g, field, value, msel_validate_embed_bwd(&a, &x, ws, need), want)
    G(dout, NULL, MSEL_ERR_NULL);
    G(dweight, NULL, MSEL_ERR_NULL);
    G(dweight, (float *)g.dout, MSEL_ERR_ALIAS);
    G(dweight, (float *)ws, MSEL_ERR_ALIAS);
    G(dout, (char *)g.dout + 8, MSEL_ERR_ALIGN);
    for (int64_t v = 1; v <= 1 << 29; v = v * 6 + 1)
        for (int64_t t = 1; t <= 1 << 30; t = t * 11 + 1)
            if (t * 64 <= (int64_t)1 << 40 && v * 64 <= (int64_t)1 << 40)
                WITH(msel_embed_args, a, vocab, (int32_t)v,
                     (x.tokens = t, msel_embed_bwd_workspace_bytes(&x) > 0), 1);
#undef N
#undef G
}

static void grads(void) {
    enum { COUNT = 300 };
    msel_tensor *t = malloc(COUNT * sizeof *t), *o = malloc(COUNT * sizeof *o);
    for (int i = 0; i < COUNT; ++i) {
        memset(&t[i], 0, sizeof t[i]);
        t[i].numel = (int64_t)i * i * 37;
        t[i].dtype = i % 2 ? MSEL_BF16 : MSEL_F32;
        t[i].data = i == 0 ? NULL : fake();
        o[i] = t[i];
        o[i].data = i == 0 ? NULL : fake();
    }
    msel_grad_args a;
    memset(&a, 0, sizeof a);
    a.abi_version = MSEL_ABI_VERSION;
    a.count = COUNT;
    a.tensors = t;
    a.outs = o;
    a.max_norm = 1.0f;
    a.eps = 1e-6f;
    a.norm = fake();
    void *ws = fake();
    const size_t need = msel_grad_workspace_bytes(&a);
    EXPECT(need > 0, 1);
    EXPECT(msel_grad_workspace_bytes(NULL), 0);
    EXPECT(msel_validate_grad_clip(&a, ws, need), MSEL_OK);
    EXPECT(msel_validate_grad_norm(&a, ws, need), MSEL_OK);
    EXPECT(msel_grad_clip(&a, ws, need - 1, NULL), MSEL_ERR_WORKSPACE);
    EXPECT(msel_grad_norm(&a, NULL, 0, NULL), MSEL_ERR_WORKSPACE);
    EXPECT(msel_grad_norm(NULL, ws, need, NULL), MSEL_ERR_NULL);
#define N(field, value, want) \
    WITH(msel_grad_args, a, field, value, msel_grad_clip(&x, ws, need, NULL), want)
    N(abi_version, 0, MSEL_ERR_VERSION);
    N(count, -1, MSEL_ERR_SHAPE);
    N(count, INT32_MAX, MSEL_ERR_SHAPE);
    N(tensors, NULL, MSEL_ERR_NULL);
    N(outs, NULL, MSEL_ERR_NULL);
    N(norm, NULL, MSEL_ERR_NULL);
    N(max_norm, -1.0f, MSEL_ERR_SHAPE);
    N(max_norm, NAN, MSEL_ERR_SHAPE);
    N(eps, -1.0f, MSEL_ERR_SHAPE);
    N(norm, (float *)t[5].data, MSEL_ERR_ALIAS);
    N(norm, (float *)o[5].data, MSEL_ERR_ALIAS);
#define T(list, i, field, value, want)                         \
    do {                                                       \
        const msel_tensor keep = list[i];                      \
        list[i].field = value;                                 \
        EXPECT(msel_grad_clip(&a, ws, need, NULL), want);      \
        list[i] = keep;                                        \
    } while (0)
    T(t, 299, numel, -1, MSEL_ERR_SHAPE);
    T(t, 299, numel, INT64_MAX, MSEL_ERR_SHAPE);
    T(t, 1, data, NULL, MSEL_ERR_NULL);
    T(t, 2, data, (char *)t[2].data + 2, MSEL_ERR_ALIGN);
    T(t, 3, dtype, 9, MSEL_ERR_DTYPE);
    T(t, 4, reserved, 1, MSEL_ERR_VERSION);
    T(t, 6, data, ws, MSEL_ERR_ALIAS);
    T(o, 299, numel, 5, MSEL_ERR_SHAPE);
    T(o, 1, dtype, MSEL_F32, MSEL_ERR_DTYPE);
    T(o, 1, data, NULL, MSEL_ERR_NULL);
    T(o, 7, data, ws, MSEL_ERR_ALIAS);
    /* no tensors at all, and totals at the limit */
    a.count = 0;
    EXPECT(msel_grad_workspace_bytes(&a) > 0, 1);
    EXPECT(msel_validate_grad_clip(&a, ws, msel_grad_workspace_bytes(&a)), MSEL_OK);
    a.count = 2;
    t[1].numel = (int64_t)1 << 40;
    t[0].numel = 0;
    EXPECT(msel_grad_workspace_bytes(&a) > 0, 1);
    t[0] = t[1];
    EXPECT(msel_grad_workspace_bytes(&a), 0);
    free(t);
    free(o);
}

int main(void) {
    norm();
    gated();
    embed();
    grads();
    if (failures) {
        fprintf(stderr, "%d expectations failed\n", failures);
        return 1;
    }
    printf("all checks passed\n");
    return 0;
}
