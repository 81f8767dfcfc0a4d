// Launch plans of the paged-cache attention against its workspace query, on the CPU: a workspace
// of the query's size for one length serves every shorter one, the query grows with the length,
// and a plan's need is that of its partial rows. Linked against the library's host code; nothing
// is launched. Prints the first shape that fails and exits non-zero.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <random>

#include "attn.h"
#include "bdssm.h"

using namespace bdssm;

namespace {

struct Shape {
    int dtype, headdim, batch, kv, group, tokens, block, window, sinks;
};

AttnPlan plan_of(const Shape &s, int len)
{
    AttnArgs a{};
    a.batch = s.batch, a.H = s.kv * s.group, a.KV = s.kv;
    a.block_len = s.tokens, a.max_len = len;
    a.block = s.block, a.window = s.window, a.sinks = s.sinks;
    return attn_plan(a, s.headdim, s.dtype == BDSSM_BF16);
}

size_t query(const Shape &s, int len)
{
    const bdssm_attn_dims d = {s.batch, s.kv * s.group, s.kv, s.headdim, s.dtype, 64};
    const bdssm_attn_mask m = {0.125f, s.block, s.window, s.sinks};
    return bdssm_attn_step_workspace(&d, s.tokens, len, &m);
}

int fail(const char *what, const Shape &s, int len, size_t have, size_t want)
{
    std::printf("%s: dtype %d, %d x %d tokens, %d heads over %d of %d, block %d, window %d + %d, length %d: %zu, %zu\n",
                what, s.dtype, s.batch, s.tokens, s.kv * s.group, s.kv, s.headdim, s.block, s.window, s.sinks, len, have,
                want);
    return 1;
}

bdssm_status call_step(const Shape &s, int len, size_t bytes)
{
    auto at = [](int i) { return reinterpret_cast<void *>((uintptr_t{1} << 45) + (static_cast<uintptr_t>(i) << 41)); };
    const int64_t qw = static_cast<int64_t>(s.kv) * s.group * s.headdim, kw = static_cast<int64_t>(s.kv) * s.headdim;
    const int pages = (len + 63) / 64;
    const bdssm_attn_dims d = {s.batch, s.kv * s.group, s.kv, s.headdim, s.dtype, 64};
    const bdssm_attn_mask m = {0.125f, s.block, s.window, s.sinks};
    const bdssm_attn_chunk c = {at(0), at(1), at(2), qw, kw, kw, static_cast<int64_t>(s.batch) * s.tokens, nullptr, s.tokens};
    const bdssm_kv_cache k = {at(3), at(4), static_cast<int32_t *>(at(5)), static_cast<int32_t *>(at(6)), 1, pages, len};
    return bdssm_attn_step(&d, &c, &k, &m, at(7), at(8), bytes, nullptr);
}

int check(const Shape &s, int longest, int step)
{
    size_t most = 0, before = 0;
    for (int64_t len = 0; len <= longest; len += step) {
        const int n = static_cast<int>(len);
        const AttnPlan p = plan_of(s, n);
        const size_t rows = static_cast<size_t>(s.batch) * s.kv * s.group * s.tokens * p.nsplit;
        const size_t need = p.nsplit == 1 ? 0 : (rows * 8 + 255) / 256 * 256 + rows * s.headdim * 4;
        if (p.ws_bytes != need)
            return fail("a plan's need is not its partial rows", s, n, p.ws_bytes, need);
        if (need > 0 && call_step(s, n, need - 1) != BDSSM_ERR_WORKSPACE)
            return fail("a step takes a byte less than its plan needs", s, n, need - 1, need);
        most = std::max(most, need);
        const size_t q = query(s, n);
        if (q < most)
            return fail("the query is below a shorter length's need", s, n, q, most);
        if (q < before)
            return fail("the query falls", s, n, q, before);
        before = q;
    }
    return 0;
}

}  // namespace

int main()
{
    // few units of many row tiles, dealt to the XCDs in parts and walked tile by tile (the launch of
    // a prompt): shapes that tests on the GPU take for it
    for (const Shape &s : {Shape{BDSSM_BF16, 64, 33, 1, 64, 33, 0, 0, 0}, Shape{BDSSM_BF16, 128, 33, 1, 64, 33, 32, 0, 0}}) {
        const AttnPlan p = plan_of(s, 500);
        if (p.sub < 2 || p.rt_fast || p.nsplit != 1)
            return fail("not a prompt's launch", s, 500, p.sub, p.rt_fast);
    }
    const Shape known[] = {
        {BDSSM_BF16, 64, 1, 8, 5, 32, 0, 0, 0},    {BDSSM_BF16, 64, 1, 4, 6, 32, 0, 0, 0},
        {BDSSM_BF16, 128, 2, 4, 5, 1024, 0, 0, 0}, {BDSSM_BF16, 64, 1, 4, 6, 1, 0, 0, 0},
        {BDSSM_BF16, 128, 1, 4, 5, 8192, 32, 0, 0}, {BDSSM_F32, 64, 2, 16, 1, 1031, 1, 512, 0},
    };
    for (const Shape &s : known)
        if (check(s, 1024, 1) || check(s, 70000, 32))
            return 1;
    std::mt19937 g(11);
    auto pick = [&](std::initializer_list<int> v) { return v.begin()[g() % v.size()]; };
    auto spread = [&](int top) { return 1 + static_cast<int>(g() % (1u << g() % (32 - __builtin_clz(top)))) % top; };
    for (int i = 0; i < 400; ++i) {
        Shape s = {pick({BDSSM_F32, BDSSM_BF16}), pick({64, 128}), spread(256), spread(32), pick({1, 1, 2, 3, 5, 8, 33}),
                   spread(4096), pick({0, 0, 1, 32, 1000}), 0, 0};
        if (g() % 3 == 0)
            s.window = spread(8192), s.sinks = pick({0, 4, 200});
        if (s.kv * s.group > 512)
            s.group = 1;
        if (check(s, 1500, 1 + static_cast<int>(g() % 17)) || check(s, 300000, 2000 + static_cast<int>(g() % 500)))
            return 1;
    }
    std::puts("ok");
    return 0;
}
