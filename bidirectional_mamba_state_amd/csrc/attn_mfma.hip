// Attention of a chunk over a paged cache: launch plans, and the launch of the kernels of
// attn_kernel.h for plain scores (attn_ranged.hip, attn_capped.hip and attn_exact.hip launch the others).
#include <algorithm>
#include <cmath>

#include "attn_kernel.h"

namespace bdssm {
namespace {

// Launch plan and workspace of one kernel shape.
template <typename T, int D, int WM, int WK, int TK, int WPE>
struct Planner {
    using C = AttnCfg<T, D, WM, WK, TK>;
    static constexpr bool f32 = sizeof(T) == 4;
    // Ranges: the number with which an XCD's workgroups take the fewest tiles one after the
    // other. A workgroup costs tiles beside its own: its start and first copies, and where
    // the keys are split its partial rows and their join. The rounds are whole, and streams
    // being of unequal lengths the last one ends half a workgroup late; only row
    // tiles that come longest first (`graded`) end together.
    // float32 products fill a CU's matrix cores with one workgroup, so that two take turns;
    // with bf16 all that fit run together (64 streams of 16-32K tokens, 768 rows: 1495 us
    // whole, 1254 in the four that it takes; 564 float32 rows on 33,169 tokens: 370 us in 17,
    // 285 in 25; a prompt of 8,192: 1020 us whole, 1077 in two; 4,096 tokens of 20 heads of 128,
    // window 512 without order: 142 us whole, 159 in two).
    // A range has two tiles at least, so that copies overlap products (192 rows on 532 keys:
    // 13.5 us in ranges of four tiles, 11.7); a float32 tile takes longer than its start and
    // may stand alone (32 x 6 rows on 1,032 keys: 26.7 us in ranges of four, 15.9). A second
    // launch costs as much as eight bf16 tiles (24 rows on 259 keys: 8.4 us whole, 11.7 in two).
    static constexpr int64_t kStart = f32 ? 2 : 3, kSplit = f32 ? 1 : 8;
    // At most 64 ranges: with four KV heads or more these fill the GPU (131,072 keys of headdim 128,
    // one token of 24 heads over 4: 49 us, 53 us with up to 128). A stream of one or two KV heads
    // alone would take more: one token of 6 heads over 1 on 131,072 keys of headdim 64 33 us, 24 us
    // with up to 128, 20 us with up to 256.
    static constexpr int kMostRanges = 64;
    const AttnArgs &a;
    int64_t R, units, slots;  // rows per unit, (stream, KV head) pairs, workgroups of an XCD at a time
    int nrt;
    explicit Planner(const AttnArgs &args)
        : a(args), R(static_cast<int64_t>(a.block_len) * (a.H / a.KV)), units(static_cast<int64_t>(a.batch) * a.KV),
          slots(std::max(1, device_cus() / 8) * (f32 ? 1 : 4 * WPE / C::NW)), nrt(static_cast<int>((R + C::RT - 1) / C::RT))
    {
    }
    // keys of one row tile, at most; a window only looks back, and ahead of a row tile are the
    // rest of its last row's block, or the whole chunk (`ahead`)
    int64_t span() const { return std::min<int64_t>(a.block_len, (C::RT + a.H / a.KV - 1) / (a.H / a.KV)); }
    int64_t back() const { return static_cast<int64_t>(a.window) + a.sinks + span(); }
    int64_t ahead() const { return std::min<int64_t>(a.block_len - span(), a.block ? a.block - 1 : INT_MAX); }
    int64_t tiles(int64_t max_len) const
    {
        int64_t keys = max_len + a.block_len;
        if (a.window)
            keys = std::min(keys, back() + ahead() + TK);
        return (keys + TK - 1) / TK;
    }
    bool ranged() const { return a.score.ranged(); }
    // row tiles of rows with ranges are sorted where they take more than one round
    size_t order_bytes() const
    {
        return ranged() && units * nrt > 8 * slots ? static_cast<size_t>((static_cast<int64_t>(a.batch) * nrt * 4 + 255) / 256 * 256)
                                                   : 0;
    }
    int64_t candidates(int64_t tiles) const  // 1 to so many ranges come into question
    {
        // rows with ranges of their own may see few of the keys (documents packed into a chunk): their
        // keys are cut only as far as it takes to fill the GPU once
        const int64_t fill = ranged() ? (8 * slots + units * nrt - 1) / (units * nrt) : kMostRanges;
        return std::max<int64_t>(1, std::min({static_cast<int64_t>(kMostRanges), fill, f32 ? tiles : (tiles + 1) / 2,
                                              kMaxGroups / 8 / (units * nrt)}));
    }
    AttnPlan deal(int64_t ns) const  // the parts of a launch with ns ranges
    {
        AttnPlan p{};
        const int64_t all = units * ns;
        p.nrt = nrt;
        p.nsplit = static_cast<int>(ns);
        p.sub = static_cast<int>(all >= 64 ? 1 : std::min<int64_t>(nrt, (64 + all - 1) / all));
        p.nrt_sub = (nrt + p.sub - 1) / p.sub;
        p.units = static_cast<int>(all * p.sub);
        p.per_xcd = (p.units + 7) / 8;
        return p;
    }
    int64_t per_xcd(int64_t ns) const  // workgroups of an XCD
    {
        const AttnPlan p = deal(ns);
        return static_cast<int64_t>(p.per_xcd) * p.nrt_sub;
    }
    // The lengths for which a unit's row tiles come longest first and end together: a prompt in
    // order, and a window without order where most of a row tile's keys are ahead of it and the
    // tiles take more than one round. With float32 the latter still gains from whole rounds (2 x
    // 1,031 tokens of 16 heads, window 512: 152 us whole, 103 in two).
    struct Lengths {
        int64_t from, to;  // [from, to)
    };
    Lengths graded() const
    {
        if (a.block)
            return {0, 2ll * a.block_len};
        if (!f32 && a.window && per_xcd(1) > slots && 2 * back() < back() + ahead() + TK)
            return {std::max<int64_t>(0, 2 * back() + 1 - a.block_len), INT64_MAX};
        return {0, 0};
    }
    AttnPlan plan() const
    {
        const int64_t nt = tiles(a.max_len), top = candidates(nt);
        const bool by_length = a.max_len >= graded().from && a.max_len < graded().to;
        int64_t ns = 1, best = INT64_MAX;
        for (int64_t x = 1; x <= top; ++x) {
            const int64_t per = (nt + x - 1) / x, each = per + kStart + (x > 1 ? kSplit : 0), here = per_xcd(x);
            const int64_t cost = by_length && here > slots ? 2 * here * each / slots : 2 * ((here + slots - 1) / slots) * each + per;
            if (cost < best)
                best = cost, ns = x;
        }
        AttnPlan p = deal(ns);
        p.rt_fast = p.nrt_sub <= 4;
        p.by_inner = Divisor(p.rt_fast ? p.nrt_sub : p.per_xcd);
        p.by_units = Divisor(units * ns);
        p.by_kv = Divisor(a.KV);
        p.by_split = Divisor(ns);
        p.groups = 8ll * p.per_xcd * p.nrt_sub;
        p.ml_bytes = ns > 1 ? ml_bytes(ns) : 0;
        p.order_bytes = order_bytes();
        p.ws_bytes = (ns > 1 ? bytes(ns) : 0) + p.order_bytes;
        for (int64_t keys = (static_cast<int64_t>(a.max_len) + a.block_len) / TK; keys >> p.order_shift >= 1024;)
            ++p.order_shift;
        return p;
    }
    size_t ml_bytes(int64_t ns) const { return static_cast<size_t>((units * R * ns * 8 + 255) / 256 * 256); }
    size_t bytes(int64_t ns) const { return ml_bytes(ns) + static_cast<size_t>(units * R * ns) * D * 4; }
    // An upper bound of the ranges that plan() takes for any length whose tiles are lo to hi
    // (`least` or more; exact for half of the shapes, a third above for one in ten). In tiles per
    // range p = ceil(tiles / x), x ranges cost per p + fixed, and y < x ranges
    // per' ceil(tiles / y) + fixed' <= per' (p x + y - 1) / y + fixed'. x is taken only if it
    // costs less than every such y: each leaves an interval of p, and x is out where none is left.
    int64_t most_ranges(bool by_length, int64_t lo, int64_t hi, int64_t least) const
    {
        struct {
            double per, fixed;
        } cost[kMostRanges + 1];
        const int top = static_cast<int>(candidates(hi));
        for (int x = 1; x <= top; ++x) {
            const int64_t here = per_xcd(x);
            const double turns = by_length && here > slots ? 2. * here / slots : 2. * ((here + slots - 1) / slots);
            cost[x] = {by_length && here > slots ? turns : turns + 1, turns * (kStart + (x > 1 ? kSplit : 0))};
        }
        for (int x = top; x > least; --x) {
            double from = std::max<double>((lo + x - 1) / x, f32 ? 1 : 2), to = (hi + x - 1) / x;
            for (int y = x - 1; y > 0 && from <= to; --y) {
                const double slope = cost[x].per - cost[y].per * x / y;
                const double room = cost[y].fixed - cost[x].fixed + cost[y].per * (y - 1) / y;  // slope p < room
                if (slope > 0)
                    to = std::min(to, std::floor(room / slope + 1e-6));
                else if (slope < 0)
                    from = std::max(from, std::ceil(room / slope - 1e-6));
                else if (room <= 0)
                    to = 0;
            }
            if (from <= to)
                return x;
        }
        return least;
    }
    // what any length up to max_len can need; SIZE_MAX: more rows than a launch has threads for
    size_t workspace() const
    {
        if (8 * per_xcd(1) > kMaxGroups)
            return SIZE_MAX;
        const Lengths g = graded();
        int64_t most = 1;
        auto lengths = [&](bool by_length, int64_t from, int64_t to) {
            to = std::min<int64_t>(to, a.max_len + 1ll);
            if (from < to)
                most = most_ranges(by_length, tiles(from), tiles(to - 1), most);
        };
        lengths(false, 0, g.from);
        lengths(true, g.from, g.to);
        lengths(false, std::max(g.from, g.to), INT64_MAX);
        return (most > 1 ? bytes(most) : 0) + order_bytes();
    }
};

struct PlanOf {
    const AttnArgs &a;
    template <typename T, int D, int WM, int WK, int TK, int WPE>
    AttnPlan operator()() const
    {
        return Planner<T, D, WM, WK, TK, WPE>(a).plan();
    }
};

struct WorkspaceOf {
    const AttnArgs &a;
    template <typename T, int D, int WM, int WK, int TK, int WPE>
    size_t operator()() const
    {
        return Planner<T, D, WM, WK, TK, WPE>(a).workspace();
    }
};

}  // namespace

AttnPlan attn_plan(const AttnArgs &a, int D, bool bf16)
{
    return by_type(a, D, bf16, PlanOf{a});
}

size_t attn_workspace(const AttnArgs &a, int D, bool bf16)
{
    return by_type(a, D, bf16, WorkspaceOf{a});
}

hipError_t launch_attn(const AttnArgs &a, int D, bool bf16, const AttnPlan &p, void *ws, hipStream_t st)
{
    return by_type(a, D, bf16, Launch<kPlain>{a, p, ws, st});
}

}  // namespace bdssm
