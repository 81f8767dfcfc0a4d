// Launch plans of attention with ranges of rows (bdssm_attn_step_ex) against its workspace query, on
// the CPU: a workspace of the query's size for one length serves every shorter one, a plan's need is
// that of its partial rows and the order of its row tiles, and without ranges everything is as in
// plain attention. Linked against the library's host code; nothing is launched.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <random>

#include "attn.h"
#include "bdssm.h"

using namespace bdssm;

namespace {

struct Shape {
    int dtype, headdim, batch, kv, group, tokens, block, window;
    bool ranged;
};

const int32_t *fake() { return reinterpret_cast<const int32_t *>(uintptr_t{1} << 40); }

AttnPlan plan_of(const Shape &s, int len)
{
    AttnArgs a{};
    a.batch = s.batch, a.H = s.kv * s.group, a.KV = s.kv;
    a.block_len = s.tokens, a.max_len = len;
    a.block = s.block, a.window = s.window;
    a.score.first = s.ranged ? fake() : nullptr;
    return attn_plan(a, s.headdim, s.dtype == BDSSM_BF16);
}

size_t query(const Shape &s, int len)
{
    const bdssm_attn_dims d = {s.batch, s.kv * s.group, s.kv, s.headdim, s.dtype, 64};
    const bdssm_attn_mask m = {0.125f, s.block, s.window, 0};
    const bdssm_attn_scores x = {5.f, nullptr, nullptr, s.ranged ? fake() : nullptr, nullptr};
    return bdssm_attn_step_ex_workspace(&d, s.tokens, len, &m, &x);
}

size_t plain(const Shape &s, int len)
{
    const bdssm_attn_dims d = {s.batch, s.kv * s.group, s.kv, s.headdim, s.dtype, 64};
    const bdssm_attn_mask m = {0.125f, s.block, s.window, 0};
    return bdssm_attn_step_workspace(&d, s.tokens, len, &m);
}

int fail(const char *what, const Shape &s, int len, size_t have, size_t want)
{
    std::printf("%s: dtype %d, %d x %d tokens, %d heads over %d of %d, block %d, window %d, ranged %d, length %d: %zu, %zu\n",
                what, s.dtype, s.batch, s.tokens, s.kv * s.group, s.kv, s.headdim, s.block, s.window, s.ranged, len, have, want);
    return 1;
}

int check(const Shape &s, int longest, int step)
{
    size_t before = 0;
    for (int64_t len = 0; len <= longest; len += step) {
        const int n = static_cast<int>(len);
        const AttnPlan p = plan_of(s, n);
        const size_t rows = static_cast<size_t>(s.batch) * s.kv * s.group * s.tokens * p.nsplit;
        const size_t part = p.nsplit == 1 ? 0 : (rows * 8 + 255) / 256 * 256 + rows * s.headdim * 4;
        const size_t order = p.order_bytes ? (static_cast<size_t>(s.batch) * p.nrt * 4 + 255) / 256 * 256 : 0;
        if (p.order_bytes != order || p.ws_bytes != part + order)
            return fail("a plan's need is not its partial rows and its order", s, n, p.ws_bytes, part + order);
        if (!s.ranged && order)
            return fail("rows without ranges are sorted", s, n, order, 0);
        const int64_t keys = len + s.tokens;
        if ((keys / 32 >> p.order_shift) >= 4096 || p.order_shift > 26)
            return fail("classes of row tiles are too coarse or too many", s, n, p.order_shift, 0);
        const size_t q = query(s, n);
        if (q < p.ws_bytes || q < before)
            return fail("the query is below a shorter length's need", s, n, q, std::max(before, p.ws_bytes));
        if (!s.ranged && q != plain(s, n))
            return fail("without ranges the query is not plain attention's", s, n, q, plain(s, n));
        before = q;
    }
    return 0;
}

}  // namespace

int main()
{
    // shapes that tests on the GPU take for sorted row tiles, and for ranges of keys
    for (const Shape &s : {Shape{BDSSM_BF16, 64, 33, 8, 1, 300, 0, 0, true}, Shape{BDSSM_BF16, 128, 22, 8, 1, 300, 1, 0, true},
                           Shape{BDSSM_F32, 64, 11, 8, 1, 300, 1, 0, true}})
        if (plan_of(s, 200).order_bytes == 0)
            return fail("not sorted", s, 200, 0, 0);
    for (int dtype : {BDSSM_F32, BDSSM_BF16})
        if (plan_of(Shape{dtype, 64, 1, 1, 2, 3, 0, 0, true}, 3000).nsplit == 1)
            return fail("not cut", Shape{dtype, 64, 1, 1, 2, 3, 0, 0, true}, 3000, 1, 2);
    std::mt19937 g(7);
    auto pick = [&](std::initializer_list<int> v) { return v.begin()[g() % v.size()]; };
    auto spread = [&](int top) { return 1 + static_cast<int>(g() % (1u << g() % (32 - __builtin_clz(top)))) % top; };
    for (int i = 0; i < 300; ++i) {
        Shape s = {pick({BDSSM_F32, BDSSM_BF16}), pick({64, 128}), spread(256), spread(32), pick({1, 1, 2, 3, 5, 8, 33}),
                   spread(8192), pick({0, 0, 1, 32, 1000}), g() % 3 == 0 ? spread(8192) : 0, g() % 4 != 0};
        if (s.kv * s.group > 512)
            s.group = 1;
        if (check(s, 1500, 1 + static_cast<int>(g() % 17)) || check(s, 300000, 2000 + static_cast<int>(g() % 500)))
            return 1;
    }
    if (check({BDSSM_BF16, 64, 1, 1, 1, 1, 0, 0, true}, 2000000000, 99999999))
        return 1;
    std::puts("ok");
    return 0;
}
