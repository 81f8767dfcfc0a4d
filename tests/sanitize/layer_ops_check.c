/*
 * Calls the norm and attention entry points of include/bdssm.h with argument sets that
 * validation must reject (or that have nothing to do), and the workspace query over many
 * shapes, so that a build of norm.hip and attn.hip with AddressSanitizer and
 * UndefinedBehaviorSanitizer on the host side checks their validation and planning. Nothing
 * here reaches a kernel or needs a GPU. Exits non-zero if a call returns an unexpected status.
 */
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "bdssm.h"

#define P(v) ((void *)(uintptr_t)(v))
#define EXPECT(call, want)                                                           \
    do {                                                                             \
        const int rc_ = (int)(call);                                                 \
        if (rc_ != (want)) {                                                         \
            fprintf(stderr, "%s: got %d (%s), want %d\n", #call, rc_, bdssm_status_str(rc_), (int)(want)); \
            return 1;                                                                \
        }                                                                            \
    } while (0)

int main(void)
{
    const uintptr_t base = (uintptr_t)1 << 40, gb = (uintptr_t)1 << 30;
    /* norms */
    bdssm_norm_dims n = {8, 100, 2, 3, BDSSM_NORM_RMS, BDSSM_F32, BDSSM_BF16, 1e-5f};
    const float *w = (const float *)P(base + 2 * gb);
    EXPECT(bdssm_gated_norm(NULL, P(base), P(base), 100, w, 0, P(base), NULL), BDSSM_ERR_NULL);
    EXPECT(bdssm_gated_norm(&n, P(base), NULL, 100, w, 0, P(base), NULL), BDSSM_ERR_NULL);
    EXPECT(bdssm_gated_norm(&n, P(base), P(base + gb), 99, w, 0, P(base + 3 * gb), NULL), BDSSM_ERR_SHAPE);
    EXPECT(bdssm_gated_norm(&n, P(base), P(base + gb), INT64_MAX / 1024, w, 0, P(base + gb + 2), NULL), BDSSM_ERR_ALIAS);
    n.groups = 1;
    bdssm_residual r = {P(base), P(base + gb), NULL, w, P(base + 4 * gb), NULL, NULL, 100, 1.f};
    EXPECT(bdssm_residual_norm(&n, NULL, P(base), P(base), NULL), BDSSM_ERR_NULL);
    EXPECT(bdssm_residual_norm(&n, &r, NULL, NULL, NULL), BDSSM_ERR_NULL);
    EXPECT(bdssm_residual_norm(&n, &r, P(base + 64), NULL, NULL), BDSSM_ERR_ALIAS);
    n.rows = INT64_MAX;
    EXPECT(bdssm_residual_norm(&n, &r, P(base), NULL, NULL), BDSSM_ERR_UNSUPPORTED);
    n.rows = 0;
    EXPECT(bdssm_residual_norm(&n, &r, P(base), NULL, NULL), BDSSM_OK);
    /* attention */
    bdssm_attn_dims d = {2, 4, 2, 64, BDSSM_BF16, 16};
    bdssm_attn_chunk c = {P(base), P(base + gb), P(base + 2 * gb), 256, 128, 128, 16, NULL, 8};
    bdssm_kv_cache k = {P(base + 3 * gb), P(base + 4 * gb), (const int32_t *)P(base + 5 * gb),
                        (const int32_t *)P(base + 6 * gb), 10, 4, 64};
    bdssm_attn_mask m = {0.125f, 0, 0, 0};
    void *out = P(base + 8 * gb), *ws = P(base + 9 * gb);
    EXPECT(bdssm_attn_step(NULL, &c, &k, &m, out, ws, gb, NULL), BDSSM_ERR_NULL);
    EXPECT(bdssm_attn_step(&d, &c, &k, &m, NULL, ws, gb, NULL), BDSSM_ERR_NULL);
    EXPECT(bdssm_attn_step(&d, &c, &k, &m, (void *)c.q, ws, gb, NULL), BDSSM_ERR_ALIAS);
    m.scale = NAN;
    EXPECT(bdssm_attn_step(&d, &c, &k, &m, out, ws, gb, NULL), BDSSM_ERR_UNSUPPORTED);
    m.scale = 0.125f;
    c.block_len = INT_MAX;
    EXPECT(bdssm_attn_step(&d, &c, &k, &m, out, ws, gb, NULL), BDSSM_ERR_SHAPE);
    c.starts = (const int32_t *)P(base + 7 * gb);
    EXPECT(bdssm_attn_step(&d, &c, &k, &m, out, ws, gb, NULL), BDSSM_ERR_UNSUPPORTED);
    EXPECT(bdssm_kv_append(&d, &c, &k, NULL, NULL), BDSSM_ERR_UNSUPPORTED);
    c.block_len = 8;
    k.max_pages = INT_MAX;
    k.max_len = INT_MAX;
    EXPECT(bdssm_attn_step(&d, &c, &k, &m, out, ws, gb, NULL), BDSSM_ERR_UNSUPPORTED);
    k.max_pages = 100000;
    k.max_len = 1000000;
    EXPECT(bdssm_attn_step(&d, &c, &k, &m, out, NULL, 0, NULL), BDSSM_ERR_WORKSPACE);
    EXPECT(bdssm_attn_step(&d, &c, &k, &m, out, P(base + 2 * gb), gb, NULL), BDSSM_ERR_ALIAS);
    EXPECT(bdssm_kv_append(&d, &c, &k, (int32_t *)k.lens, NULL), BDSSM_ERR_ALIAS);
    /* the workspace of any shape is a number, and covers the ranges' rows */
    for (int dt = 0; dt < 2; ++dt)
        for (int hd = 64; hd <= 128; hd += 64)
            for (int g = 1; g <= 64; g *= 4)
                for (int64_t T = 1; T < INT_MAX / 2; T *= 37)
                    for (int64_t L = 0; L < INT_MAX / 2; L = 3 * L + 1)
                        for (int win = 0; win < 3; ++win) {
                            bdssm_attn_dims x = {3, 2 * g, 2, hd, dt, 64};
                            bdssm_attn_mask y = {1.f, win, win == 2 ? INT_MAX : win * 100, win == 2 ? INT_MAX : win};
                            const size_t b = bdssm_attn_step_workspace(&x, (int32_t)T, (int32_t)L, &y);
                            if (b != SIZE_MAX && b % 16 != 0)
                                return 1;
                        }
    puts("layer operators sanitizer run: ok");
    return 0;
}
