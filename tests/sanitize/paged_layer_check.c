/*
 * Calls the rotary, scored-attention and page entry points of include/bdssm.h with argument sets
 * that validation must reject (or that have nothing to do), the workspace queries over many
 * shapes and the table of rotary frequencies, so that a build of rotary.hip, pages.hip, attn.hip
 * and attn_mfma.hip with AddressSanitizer and UndefinedBehaviorSanitizer on the host side checks
 * their host code. Nothing here reaches a kernel or needs a GPU. Exits non-zero if a call returns
 * an unexpected status.
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
    bdssm_attn_dims d = {2, 4, 2, 64, BDSSM_BF16, 16};
    bdssm_attn_chunk c = {P(base), P(base + gb), P(base + 2 * gb), 256, 128, 128, 16, NULL, 8};
    bdssm_kv_cache k = {P(base + 3 * gb), P(base + 4 * gb), (const int32_t *)P(base + 5 * gb),
                        (const int32_t *)P(base + 6 * gb), 10, 4, 64};
    bdssm_attn_mask m = {0.125f, 0, 0, 0};
    /* scores */
    bdssm_attn_scores s = {5.f, (const float *)P(base + 10 * gb), (const int32_t *)P(base + 11 * gb),
                           (const int32_t *)P(base + 12 * gb), (const int32_t *)P(base + 13 * gb)};
    void *out = P(base + 8 * gb), *ws = P(base + 9 * gb);
    EXPECT(bdssm_attn_step_ex(&d, &c, &k, &m, NULL, out, ws, gb, NULL), BDSSM_ERR_NULL);
    EXPECT(bdssm_attn_step_ex(&d, &c, &k, &m, &s, P(base + 12 * gb), ws, gb, NULL), BDSSM_ERR_ALIAS);
    const float caps[] = {-1.f, NAN, INFINITY, 1e-45f, 1e-39f, 3e38f};
    for (unsigned i = 0; i < sizeof caps / sizeof *caps; ++i) {
        s.cap = caps[i];
        EXPECT(bdssm_attn_step_ex(&d, &c, &k, &m, &s, out, ws, gb, NULL), BDSSM_ERR_UNSUPPORTED);
    }
    for (float cap = 1e-30f; cap < 1e30f; cap *= 10.f) {  /* any that is taken, up to the overlap check */
        s.cap = cap;
        EXPECT(bdssm_attn_step_ex(&d, &c, &k, &m, &s, (void *)c.q, ws, gb, NULL), BDSSM_ERR_ALIAS);
    }
    s.cap = 0.f;
    k.max_pages = 100000;
    k.max_len = 1000000;
    EXPECT(bdssm_attn_step_ex(&d, &c, &k, &m, &s, out, NULL, 0, NULL), BDSSM_ERR_WORKSPACE);
    k.max_pages = 4;
    k.max_len = 64;
    for (int dt = 0; dt < 2; ++dt)
        for (int hd = 64; hd <= 128; hd += 64)
            for (int g = 1; g <= 64; g *= 4)
                for (int64_t T = 1; T < INT_MAX / 2; T *= 37)
                    for (int64_t L = 0; L < INT_MAX / 2; L = 3 * L + 1) {
                        bdssm_attn_dims x = {3, 2 * g, 2, hd, dt, 64};
                        bdssm_attn_mask y = {1.f, 1, 0, 0};
                        const size_t b = bdssm_attn_step_ex_workspace(&x, (int32_t)T, (int32_t)L, &y, &s);
                        if (b != SIZE_MAX && b % 16 != 0)
                            return 1;
                    }
    /* rotary */
    uint64_t turns[256];
    for (int kind = -1; kind <= 4; ++kind)
        for (int dim = -2; dim <= 516; dim += 2) {
            bdssm_rotary_freqs f = {dim, kind, 10000., 8., 4096, 1., 32.};
            const int bad = kind < 0 || kind > 3 || (kind == 2 && dim == 2);
            EXPECT(bdssm_rotary_turns(&f, turns), dim < 2 || dim > 512 ? BDSSM_ERR_SHAPE : bad ? BDSSM_ERR_UNSUPPORTED : BDSSM_OK);
        }
    bdssm_rotary_freqs f = {512, BDSSM_ROTARY_LINEAR, 1e300, 1e-300, 0, 0., 0.};
    EXPECT(bdssm_rotary_turns(&f, turns), BDSSM_OK);
    f.factor = 1e300;
    EXPECT(bdssm_rotary_turns(&f, turns), BDSSM_OK);
    bdssm_rotary r = {64, 0, 1.f, (const uint64_t *)P(base + 14 * gb), NULL};
    bdssm_rotary_out o = {P(base + 15 * gb), P(base + 16 * gb), 256, 128};
    EXPECT(bdssm_rotary_step(&d, &c, NULL, NULL, &o, NULL), BDSSM_ERR_NULL);
    o.q = P(base + 16);
    EXPECT(bdssm_rotary_step(&d, &c, &r, NULL, &o, NULL), BDSSM_ERR_ALIAS);
    EXPECT(bdssm_rotary_append(&d, &c, &k, &r, &o, NULL, NULL), BDSSM_ERR_ALIAS);
    o.q = P(base + 15 * gb);
    o.q_stride = INT64_MAX & ~(int64_t)7;
    EXPECT(bdssm_rotary_step(&d, &c, &r, NULL, &o, NULL), BDSSM_ERR_UNSUPPORTED);
    o.q_stride = 256;
    c.tokens = (int64_t)INT_MAX + 1;
    c.starts = (const int32_t *)P(base + 7 * gb);
    EXPECT(bdssm_rotary_step(&d, &c, &r, NULL, &o, NULL), BDSSM_ERR_UNSUPPORTED);
    c.tokens = INT_MAX;
    c.block_len = INT_MAX;
    EXPECT(bdssm_rotary_step(&d, &c, &r, NULL, &o, NULL), BDSSM_ERR_ALIAS);  /* two billion rows reach far */
    c.tokens = 16;
    c.block_len = 8;
    c.starts = NULL;
    /* pages */
    bdssm_pages_dims g = {2, 16, 100, 8};
    bdssm_pages t = {(const int32_t *)P(base), (const int32_t *)P(base + gb), (const int32_t *)P(base + 2 * gb)};
    int32_t *to = (int32_t *)P(base + 3 * gb), *uo = (int32_t *)P(base + 4 * gb), *n = (int32_t *)P(base + 5 * gb);
    int32_t *lo = (int32_t *)P(base + 7 * gb), *co = (int32_t *)P(base + 8 * gb);
    EXPECT(bdssm_pages_advance(&g, &t, NULL, 8, 0, 0, to, uo, n, ws, 0, NULL), BDSSM_ERR_WORKSPACE);
    EXPECT(bdssm_pages_advance(&g, &t, NULL, 8, -1, 0, to, uo, n, ws, gb, NULL), BDSSM_ERR_SHAPE);
    EXPECT(bdssm_pages_fork(&g, &t, lo, (int32_t *)t.table, co, uo, co + 64, n, ws, gb, NULL), BDSSM_ERR_ALIAS);
    EXPECT(bdssm_pages_compact(&g, &t, to, uo, NULL, n, ws, gb, NULL), BDSSM_ERR_NULL);
    for (int64_t b = 0; b <= 65535; b = 5 * b + 1)
        for (int64_t p = 0; p <= INT_MAX; p = 7 * p + 1) {
            bdssm_pages_dims x = {(int32_t)b, 256, (int32_t)p, 8000000};
            const size_t bytes = bdssm_pages_workspace(&x);
            if (bytes == SIZE_MAX || bytes % 16 != 0 || bytes < 8 * (size_t)p)
                return 1;
        }
    bdssm_pages_dims huge = {65535, 16, INT_MAX, 134217000};
    EXPECT(bdssm_pages_advance(&huge, &t, NULL, INT_MAX, INT_MAX, INT_MAX, to, uo, n, ws, gb, NULL), BDSSM_ERR_ALIAS);
    EXPECT(bdssm_pages_copy(&d, &k, NULL, 1, NULL), BDSSM_ERR_NULL);
    EXPECT(bdssm_pages_copy(&d, &k, (const int32_t *)k.k, INT_MAX, NULL), BDSSM_ERR_ALIAS);
    EXPECT(bdssm_pages_copy(&d, &k, NULL, 0, NULL), BDSSM_OK);
    puts("paged layer sanitizer run: ok");
    return 0;
}
