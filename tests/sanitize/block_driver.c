/*
 * Host-side code of the gated recurrence, the log probabilities and the feed-forward block under
 * AddressSanitizer and UndefinedBehaviorSanitizer.
 *
 * Built by tests/test_block_sanitizers.py with the sanitizers on the host side: checks on valid and
 * invalid arguments, workspaces sized from the smallest to the largest sizes, and entry points
 * called with invalid arguments, on which they return before any HIP call.  Device pointers are
 * fake addresses that nothing dereferences.  Exit status 0 when every expectation holds.
 */
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "msel.h"

static int failures = 0;
static uintptr_t next_addr = 0x10000000u;

static void *fake(void) {
    void *p = (void *)next_addr;
    next_addr += 0x10000000u;
    return p;
}

#define EXPECT(expr, want)                                                                       \
    do {                                                                                         \
        long long got_ = (long long)(expr);                                                      \
        if (got_ != (long long)(want)) {                                                         \
            fprintf(stderr, "%s:%d: %s = %lld, expected %lld\n", __FILE__, __LINE__, #expr, got_, \
                    (long long)(want));                                                          \
            ++failures;                                                                          \
        }                                                                                        \
    } while (0)

static const int32_t sizes[] = {1, 2, 7, 8, 9, 127, 129, 512, 513, 2048, 5000, 65536, 1 << 20, 1 << 28};
#define N_SIZES (int)(sizeof sizes / sizeof sizes[0])

static void lru(void) {
    msel_lru_args a;
    msel_lru_grads g;
    memset(&a, 0, sizeof a);
    memset(&g, 0, sizeof g);
    EXPECT(msel_lru_fwd(NULL, NULL, 0, NULL), MSEL_ERR_NULL);
    EXPECT(msel_lru_fwd(&a, NULL, 0, NULL), MSEL_ERR_VERSION);
    a.abi_version = MSEL_ABI_VERSION;
    EXPECT(msel_lru_fwd(&a, NULL, 0, NULL), MSEL_ERR_SHAPE);
    EXPECT(msel_lru_bwd(&a, &g, NULL, 0, NULL), MSEL_ERR_SHAPE);
    for (int i = 0; i < N_SIZES; ++i)
        for (int j = 0; j < N_SIZES; ++j)
            for (int k = 0; k < 3; ++k) {
                a.batch = k == 0 ? 1 : k == 1 ? 3 : 1 << 10;
                a.dim = sizes[i];
                a.seqlen = sizes[j];
                const size_t f = msel_lru_fwd_workspace_bytes(&a);
                const size_t b = msel_lru_bwd_workspace_bytes(&a);
                EXPECT(f <= b, 1);
                EXPECT(msel_lru_fwd(&a, NULL, 0, NULL) != MSEL_OK, 1); /* no pointers */
            }
    a.batch = 2;
    a.dim = 3;
    a.seqlen = 9000;
    a.x = fake();
    a.gate_a = fake();
    a.gate_x = fake();
    a.lam = fake();
    EXPECT(msel_lru_fwd(&a, NULL, 0, NULL), MSEL_ERR_NULL);
    a.out = fake();
    EXPECT(msel_lru_fwd(&a, NULL, 0, NULL), MSEL_ERR_WORKSPACE);
    EXPECT(msel_lru_bwd(&a, NULL, NULL, 0, NULL), MSEL_ERR_NULL);
    EXPECT(msel_lru_bwd(&a, &g, NULL, 0, NULL), MSEL_ERR_NULL);
    g.dout = fake();
    g.dx = fake();
    g.dgate_a = fake();
    g.dgate_x = fake();
    EXPECT(msel_lru_bwd(&a, &g, fake(), 16, NULL), MSEL_ERR_WORKSPACE);
    a.chunk_states = (float *)(void *)a.out;
    EXPECT(msel_lru_fwd(&a, NULL, 0, NULL), MSEL_ERR_ALIAS);
}

static void logprob(void) {
    static const float bad[] = {0.0f, -1.0f, NAN, INFINITY};
    msel_logprob_args a;
    msel_logprob_grads g;
    memset(&a, 0, sizeof a);
    memset(&g, 0, sizeof g);
    EXPECT(msel_logprob_fwd(NULL, NULL, 0, NULL), MSEL_ERR_NULL);
    EXPECT(msel_logprob_bwd(NULL, &g, NULL), MSEL_ERR_NULL);
    a.abi_version = MSEL_ABI_VERSION;
    EXPECT(msel_logprob_fwd(&a, NULL, 0, NULL), MSEL_ERR_SHAPE);
    a.scale = 1.0f;
    for (int i = 0; i < N_SIZES; ++i)
        for (int j = 0; j < N_SIZES; ++j)
            for (int top = 0; top <= 64; top += 16) {
                a.rows = sizes[i];
                a.vocab = sizes[j];
                a.stride = a.vocab;
                a.top = top;
                (void)msel_logprob_fwd_workspace_bytes(&a);
                EXPECT(msel_logprob_fwd(&a, NULL, 0, NULL) != MSEL_OK, 1);
            }
    a.rows = 5;
    a.vocab = 50000;
    a.stride = INT64_MAX;
    EXPECT(msel_logprob_fwd(&a, NULL, 0, NULL), MSEL_ERR_SHAPE);
    a.stride = 50000;
    a.top = 0;
    a.logits = fake();
    a.ids = fake();
    EXPECT(msel_logprob_fwd(&a, NULL, 0, NULL), MSEL_ERR_NULL);
    a.lse = fake();
    EXPECT(msel_logprob_fwd(&a, NULL, 0, NULL), MSEL_ERR_WORKSPACE);
    for (int i = 0; i < 4; ++i) {
        a.scale = bad[i];
        EXPECT(msel_logprob_fwd(&a, NULL, 0, NULL), MSEL_ERR_SHAPE);
    }
    a.scale = 1.0f;
    g.dstride = 50000;
    EXPECT(msel_logprob_bwd(&a, &g, NULL), MSEL_ERR_NULL);
    g.dlogits = (char *)a.logits + 64;
    EXPECT(msel_logprob_bwd(&a, &g, NULL), MSEL_ERR_ALIAS);
    g.dstride = INT64_MAX;
    EXPECT(msel_logprob_bwd(&a, &g, NULL), MSEL_ERR_SHAPE);
}

static void mlp(void) {
    msel_gated_mlp_args a;
    msel_gated_mlp_grads g;
    memset(&a, 0, sizeof a);
    memset(&g, 0, sizeof g);
    EXPECT(msel_gated_mlp_fwd(NULL, NULL, 0, NULL), MSEL_ERR_NULL);
    a.abi_version = MSEL_ABI_VERSION;
    EXPECT(msel_gated_mlp_fwd(&a, NULL, 0, NULL), MSEL_ERR_SHAPE);
    for (int i = 0; i < N_SIZES; ++i)
        for (int j = 0; j < N_SIZES; ++j)
            for (int k = 0; k < N_SIZES; ++k)
                for (int t = 0; t < 2; ++t) {
                    a.tokens = sizes[i];
                    a.dim = sizes[j];
                    a.hidden = sizes[k];
                    a.dtype = t;
                    const size_t f = msel_gated_mlp_fwd_workspace_bytes(&a);
                    EXPECT(f <= msel_gated_mlp_bwd_workspace_bytes(&a), 1);
                    EXPECT(msel_gated_mlp_fwd(&a, NULL, 0, NULL) != MSEL_OK, 1);
                }
    a.tokens = 100;
    a.dim = 70;
    a.hidden = 33;
    a.x = fake();
    a.w_gate = fake();
    a.w_up = fake();
    a.out = fake();
    EXPECT(msel_gated_mlp_fwd(&a, NULL, 0, NULL), MSEL_ERR_WORKSPACE);
    EXPECT(msel_gated_mlp_bwd(&a, &g, NULL, 0, NULL), MSEL_ERR_NULL);
    g.dout = fake();
    g.dx = fake();
    EXPECT(msel_gated_mlp_bwd(&a, &g, NULL, 0, NULL), MSEL_ERR_WORKSPACE);
    a.out = (void *)a.x;
    EXPECT(msel_gated_mlp_fwd(&a, NULL, 0, NULL), MSEL_ERR_ALIAS);
}

int main(void) {
    lru();
    logprob();
    mlp();
    if (failures == 0) printf("all checks passed\n");
    return failures != 0;
}
