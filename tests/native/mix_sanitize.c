/*
 * Host-side driver of the channel-mixing entry points for the sanitizer build
 * (AddressSanitizer and UndefinedBehaviorSanitizer on the host code; no kernel
 * is launched).
 *
 * It runs the validation, the choice of shapes and the workspace sizing over
 * pseudo-random descriptors from one row to the limits, and entry points with
 * arguments that are refused before any launch: bad descriptors, NULL,
 * misaligned and overlapping pointers, a short workspace.  Prints "ok <calls>"
 * and exits 0, or the first failed expectation and exits 1.
 */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../include/cnhwc.h"

static long g_calls;
static int g_fail;

#define EXPECT(cond, ...)                                                   \
    do {                                                                    \
        g_calls++;                                                          \
        if (!(cond)) {                                                      \
            if (!g_fail) {                                                  \
                printf("FAIL line %d: ", __LINE__);                         \
                printf(__VA_ARGS__);                                        \
                printf(" (last error: %s)\n", cnhwc_last_error());          \
            }                                                               \
            g_fail = 1;                                                     \
        }                                                                   \
    } while (0)

static uint64_t g_rng = 0x243f6a8885a308d3ull;
static uint64_t rnd64(void) {
    g_rng = g_rng * 6364136223846793005ull + 1442695040888963407ull;
    return g_rng >> 16;
}
/* spread over the logarithm of 1..2^bits */
static int64_t size(int bits) {
    const int b = (int)(rnd64() % (uint64_t)(bits + 1));
    return (int64_t)(1 + rnd64() % ((uint64_t)1 << b));
}

static void gated(int64_t rows, int64_t c, int64_t f, int64_t xs, int64_t ys, int act, int dtype) {
    cnhwc_gated_problem p;
    memset(&p, 0, sizeof p);
    p.rows = rows; p.c = c; p.f = f; p.x_stride = xs; p.y_stride = ys; p.act = act; p.dtype = dtype;
    for (int op = CNHWC_OP_FWD; op <= CNHWC_OP_DGRAD; ++op) {
        size_t aligned = 0, any = 0;
        char name[256], tiny[4];
        int st = cnhwc_gated_workspace_size(&p, op, 0, &aligned);
        if (st != CNHWC_OK) {
            EXPECT(st == CNHWC_INVALID_ARG && cnhwc_last_error()[0], "status %d", st);
            continue;
        }
        EXPECT(cnhwc_gated_workspace_size(&p, op, 1, &any) == CNHWC_OK, "unaligned size refused");
        EXPECT(any >= aligned, "%zu < %zu", any, aligned);
        EXPECT(cnhwc_gated_plan(&p, op, name, sizeof name) == CNHWC_OK && name[0], "plan");
        EXPECT(cnhwc_gated_plan(&p, op, tiny, sizeof tiny) == CNHWC_OK && strlen(tiny) == 3, "cut name");
        EXPECT(cnhwc_gated_plan(&p, op, NULL, 0) == CNHWC_OK, "no name");
        if (op == CNHWC_OP_DGRAD && rows > 0)
            EXPECT(aligned >= (size_t)rows * 4 * (size_t)f, "no room for dg and du: %zu", aligned);
    }
}

static void refusals(void) {
    alignas(16) static unsigned char buf[1 << 16];
    unsigned char* b = buf;
    cnhwc_layernorm_problem ln;
    memset(&ln, 0, sizeof ln);
    ln.rows = 4; ln.c = 8; ln.eps = 1e-5f;
    ln.dtype = CNHWC_F16; ln.param_dtype = CNHWC_F16;
    float* mean = (float*)(void*)(b + 8192);
    float* rstd = (float*)(void*)(b + 9216);
    EXPECT(cnhwc_layernorm_fwd(NULL, b, NULL, NULL, b + 4096, mean, rstd, NULL) == CNHWC_INVALID_ARG, "NULL problem");
    EXPECT(cnhwc_layernorm_fwd(&ln, NULL, NULL, NULL, b + 4096, mean, rstd, NULL) == CNHWC_INVALID_ARG, "NULL x");
    EXPECT(cnhwc_layernorm_fwd(&ln, b + 1, NULL, NULL, b + 4096, mean, rstd, NULL) == CNHWC_MISALIGNED, "odd x");
    EXPECT(cnhwc_layernorm_fwd(&ln, b, NULL, NULL, b + 62, mean, rstd, NULL) == CNHWC_INVALID_ARG, "y over x");
    EXPECT(cnhwc_layernorm_bwd(&ln, b, b + 512, NULL, mean, rstd, NULL, NULL, NULL, NULL, 0, NULL) ==
           CNHWC_INVALID_ARG, "nothing to compute");
    EXPECT(cnhwc_layernorm_bwd(&ln, b, b + 512, NULL, mean, rstd, b + 1024, b + 2048, b + 2560, b + 16384, 1, NULL) ==
           CNHWC_WORKSPACE_TOO_SMALL, "short workspace");
    cnhwc_gated_problem g;
    memset(&g, 0, sizeof g);
    g.rows = 100; g.c = 8; g.f = 8; g.act = CNHWC_ACT_SILU; g.dtype = CNHWC_BF16;
    EXPECT(cnhwc_gated_fwd(&g, b, b + 2048, NULL, b + 4096, NULL, 0, NULL) == CNHWC_INVALID_ARG, "NULL wu");
    EXPECT(cnhwc_gated_fwd(&g, b, b + 2048, b + 2304, b + 16, NULL, 0, NULL) == CNHWC_INVALID_ARG, "y over x");
    EXPECT(cnhwc_gated_bwd(&g, b, b + 2048, b + 4096, b + 4608, b + 8192, b + 12288, b + 12800, b + 16384, 16, NULL) ==
           CNHWC_WORKSPACE_TOO_SMALL, "short workspace");
    g.act = 9;
    EXPECT(cnhwc_gated_fwd(&g, b, b + 2048, b + 2304, b + 4096, NULL, 0, NULL) == CNHWC_INVALID_ARG, "act");
    cnhwc_dropout_problem d;
    memset(&d, 0, sizeof d);
    d.rows = 4; d.c = 8; d.p = 0.5; d.dtype = CNHWC_F32;
    EXPECT(cnhwc_dropout(&d, b, NULL, b + 16, NULL, NULL) == CNHWC_INVALID_ARG, "y over x");
    EXPECT(cnhwc_dropout(&d, b + 2, NULL, b + 4096, NULL, NULL) == CNHWC_MISALIGNED, "odd x");
    d.p = 1.5;
    EXPECT(cnhwc_dropout(&d, b, NULL, b + 4096, NULL, NULL) == CNHWC_INVALID_ARG, "p");
}

int main(void) {
    refusals();
    const int64_t big = (int64_t)1 << 20, rows = ((int64_t)1 << 31) - 1;
    gated(rows, big, big, 0, 0, CNHWC_ACT_GELU, CNHWC_F16);
    gated(rows, big, big, 2 * big, 2 * big, CNHWC_ACT_RELU, CNHWC_BF16);
    gated(rows, 1, 1, 0, 0, CNHWC_ACT_SILU, CNHWC_BF16);
    gated(1, big, big, 0, 0, CNHWC_ACT_SILU, CNHWC_BF16);
    gated(rows + 1, 8, 8, 0, 0, CNHWC_ACT_SILU, CNHWC_BF16);
    gated(INT64_MAX, INT64_MAX, INT64_MAX, INT64_MAX, INT64_MAX, 0, 0);
    gated(-1, 8, 8, 0, 0, 0, 0);
    for (int i = 0; i < 3000; ++i) {
        const int64_t c = size(20), f = size(20);
        gated(size(31) - 1, c, f, rnd64() % 3 ? 0 : c + size(10), rnd64() % 3 ? 0 : f + size(10),
              (int)(rnd64() % 5), (int)(rnd64() % 4));
    }
    cnhwc_override ov;
    memset(&ov, 0, sizeof ov);
    for (int i = 0; i < 200; ++i) {
        ov.tune = rnd64() % 2 ? 128 : 256;
        ov.split_c = (int)(rnd64() % 200);
        cnhwc_set_override(&ov);
        gated(size(31) - 1, size(20), size(20), 0, 0, CNHWC_ACT_SILU, CNHWC_F16);
    }
    cnhwc_set_override(NULL);
    for (int i = 0; i < 20000; ++i) {
        cnhwc_layernorm_problem p;
        memset(&p, 0, sizeof p);
        p.rows = (int64_t)(rnd64() << (rnd64() % 17)) >> (rnd64() % 48);
        p.c = size(32);
        p.x_stride = rnd64() % 2 ? 0 : p.c - 1 + size(33);
        p.y_stride = rnd64() % 2 ? 0 : p.c - 1 + size(33);
        p.dtype = (int)(rnd64() % 4);
        p.param_dtype = (int)(rnd64() % 4);
        size_t bytes = 1;
        const int st = cnhwc_layernorm_workspace_size(&p, &bytes);
        EXPECT(st == CNHWC_OK ? bytes % 8 == 0 : st == CNHWC_INVALID_ARG, "status %d, %zu bytes", st, bytes);
    }
    if (g_fail) return 1;
    printf("ok %ld\n", g_calls);
    return 0;
}
