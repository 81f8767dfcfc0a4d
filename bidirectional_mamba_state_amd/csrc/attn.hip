// Attention of a chunk of new tokens over a paged cache (bdssm_attn_step) and the cache's
// append (bdssm_kv_append): kernels and their host entry points.
#include <limits.h>

#include "attn.h"
#include "bdssm.h"
#include "host_checks.h"
#include "internal.h"

namespace bdssm {
namespace {

// Append: one thread copies a 16-byte piece of a token's keys and the same piece of its values
// (pieces run over [KV][D] of a token, so a wavefront reads whole lines of the chunk's rows and
// writes whole lines of a head's page). Streams along y. Bound by the copy's bytes: 5.0 TB/s both
// ways for 4 streams of 8-16K tokens of 8 heads x 128 (56 us), 3 us for one block of 32.
__global__ __launch_bounds__(256) void k_append(AttnArgs a, int *lens_out, int head_pieces, int row_pieces, int elt16)
{
    const int b = blockIdx.y;
    const AttnStream s = attn_stream(a, b);
    const int64_t held = static_cast<int64_t>(a.max_pages) << a.page_shift;
    if (lens_out && blockIdx.x == 0 && threadIdx.x == 0) {
        const int64_t end = static_cast<int64_t>(s.len) + s.n;
        lens_out[b] = static_cast<int>(end < held ? end : held);
    }
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int i = static_cast<int>(unit / row_pieces), c = static_cast<int>(unit % row_pieces);
    const int64_t j = static_cast<int64_t>(s.len) + i;
    if (i >= s.n || j >= held)
        return;
    const int pg = a.table[static_cast<int64_t>(b) * a.max_pages + (j >> a.page_shift)];
    if (pg < 0 || pg >= a.num_pages)
        return;
    const int page = 1 << a.page_shift;
    const uint4 kx = static_cast<const uint4 *>(a.k)[(s.row0 + i) * (a.k_stride / elt16) + c];
    const uint4 vx = static_cast<const uint4 *>(a.v)[(s.row0 + i) * (a.v_stride / elt16) + c];
    const int64_t to = ((static_cast<int64_t>(pg) * a.KV + c / head_pieces) * page + (j & (page - 1))) * head_pieces +
                       c % head_pieces;
    static_cast<uint4 *>(a.kp)[to] = kx;
    static_cast<uint4 *>(a.vp)[to] = vx;
}

// rows (token, head of a group) of a stream, and with them the grid's threads
bool rows_fit(const AttnArgs &a) { return static_cast<int64_t>(a.block_len) * (a.H / a.KV) <= 1 << 30; }

}  // namespace

bdssm_status check_attn_dims(const bdssm_attn_dims *d)
{
    if (!d)
        return BDSSM_ERR_NULL;
    if (d->batch < 0 || d->nheads < 1 || d->kv_heads < 1 || d->nheads % d->kv_heads != 0)
        return BDSSM_ERR_SHAPE;
    if (d->dtype != BDSSM_F32 && d->dtype != BDSSM_BF16)
        return BDSSM_ERR_UNSUPPORTED;
    if (d->headdim != 64 && d->headdim != 128)
        return BDSSM_ERR_UNSUPPORTED;
    if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128 && d->page_size != 256)
        return BDSSM_ERR_UNSUPPORTED;
    if (d->nheads > 512 || d->batch > 65535)
        return BDSSM_ERR_UNSUPPORTED;
    return BDSSM_OK;
}

namespace {

bdssm_status check_attn_mask(const bdssm_attn_mask *m)
{
    if (!m)
        return BDSSM_ERR_NULL;
    if (m->block < 0 || m->window < 0 || m->sinks < 0)
        return BDSSM_ERR_SHAPE;
    if (!(m->scale > 0.f) || m->scale - m->scale != 0.f)  // not positive, NaN or infinite
        return BDSSM_ERR_UNSUPPORTED;
    return BDSSM_OK;
}

}  // namespace

bdssm_status prepare_attn(const bdssm_attn_dims *d, const bdssm_attn_chunk *ch, const bdssm_kv_cache *ca, bool need_q,
                          bool need_kv, AttnArgs *out, AttnRanges *r)
{
    bdssm_status rc = check_attn_dims(d);
    if (rc != BDSSM_OK)
        return rc;
    if (!ch || !ca)
        return BDSSM_ERR_NULL;
    if (ch->block_len < 0 || ch->tokens < 0 || ca->num_pages < 0 || ca->max_pages < 0 || ca->max_len < 0)
        return BDSSM_ERR_SHAPE;
    if (!ch->starts && ch->tokens != static_cast<int64_t>(d->batch) * ch->block_len)
        return BDSSM_ERR_SHAPE;
    const int64_t held = static_cast<int64_t>(ca->max_pages) * d->page_size;
    if (ca->max_len > held)
        return BDSSM_ERR_SHAPE;
    if (static_cast<int64_t>(ca->max_len) + ch->block_len > kMaxPosition || ch->tokens > INT_MAX ||
        ch->q_stride > kMaxStride || ch->k_stride > kMaxStride || ch->v_stride > kMaxStride)
        return BDSSM_ERR_UNSUPPORTED;
    // an empty tensor may have no address
    if (ch->tokens > 0 && ((need_q && !ch->q) || (need_kv && !ch->k) || !ch->k != !ch->v))
        return BDSSM_ERR_NULL;
    if ((ca->num_pages > 0 && (!ca->k || !ca->v)) || (d->batch > 0 && ((ca->max_pages > 0 && !ca->table) || !ca->lens)))
        return BDSSM_ERR_NULL;
    const int e = elt(d->dtype), per16 = 16 / e;
    const int64_t qw = static_cast<int64_t>(d->nheads) * d->headdim, kw = static_cast<int64_t>(d->kv_heads) * d->headdim;
    if ((need_q && ch->q_stride < qw) || (ch->k && (ch->k_stride < kw || ch->v_stride < kw)))
        return BDSSM_ERR_SHAPE;
    if (!aligned(ch->k) || !aligned(ch->v) || !aligned(ca->k) || !aligned(ca->v) || !aligned4(ca->table) ||
        !aligned4(ca->lens) || !aligned4(ch->starts) || (need_q && (!aligned(ch->q) || ch->q_stride % per16 != 0)) ||
        (ch->k && (ch->k_stride % per16 != 0 || ch->v_stride % per16 != 0)))
        return BDSSM_ERR_ALIGN;
    auto rows = [&](const void *p, int64_t stride, int64_t width) {
        return rng(p, ch->tokens > 0 ? ((ch->tokens - 1) * stride + width) * e : 0);
    };
    const int64_t pool = static_cast<int64_t>(ca->num_pages) * d->kv_heads * d->page_size * d->headdim * e;
    *r = AttnRanges{need_q ? rows(ch->q, ch->q_stride, qw) : rng(nullptr, 0),
                    rows(ch->k, ch->k_stride, kw),
                    rows(ch->v, ch->v_stride, kw),
                    rng(ca->k, pool),
                    rng(ca->v, pool),
                    rng(ca->table, static_cast<int64_t>(d->batch) * ca->max_pages * 4),
                    rng(ca->lens, d->batch * 4ll),
                    rng(ch->starts, d->batch > 0 ? (d->batch + 1) * 4ll : 0)};
    *out = AttnArgs{};
    out->q = ch->q, out->k = ch->k, out->v = ch->v;
    out->q_stride = ch->q_stride, out->k_stride = ch->k_stride, out->v_stride = ch->v_stride;
    out->tokens = ch->tokens, out->starts = ch->starts, out->block_len = ch->block_len;
    out->kp = ca->k, out->vp = ca->v, out->table = ca->table, out->lens = ca->lens;
    out->num_pages = ca->num_pages, out->max_pages = ca->max_pages, out->max_len = ca->max_len;
    out->batch = d->batch, out->H = d->nheads, out->KV = d->kv_heads;
    out->page_shift = __builtin_ctz(d->page_size);
    return BDSSM_OK;
}

namespace {

// Fills the scoring part of a step's arguments; the ranges that its output may not overlap follow.
bdssm_status prepare_scores(const bdssm_attn_scores *s, float scale, bool bf16, AttnArgs *a, Range (&r)[4])
{
    if (!s)
        return BDSSM_ERR_NULL;
    if (!(s->cap >= 0.f) || s->cap - s->cap != 0.f)  // negative, NaN or infinite
        return BDSSM_ERR_UNSUPPORTED;
    // with bf16 the products start from the bias over the scale
    if (s->slopes && !(scale >= 0x1p-64f && scale <= 0x1p64f))
        return BDSSM_ERR_UNSUPPORTED;
    if (!aligned4(s->slopes) || !aligned4(s->prefix) || !aligned4(s->first) || !aligned4(s->last))
        return BDSSM_ERR_ALIGN;
    AttnScoring &g = a->score;
    if (s->cap > 0.f) {
        const double log2e = 1.4426950408889634074;
        g.x_per_score = static_cast<float>(static_cast<double>(scale) / s->cap);
        g.cap_log2 = static_cast<float>(s->cap * log2e);
        // both have to be ordinary numbers, or a score of zero would come out as none
        const float least = 0x1p-126f, most = 0x1p126f;
        if (!(g.x_per_score >= least && g.x_per_score <= most && g.cap_log2 >= least && g.cap_log2 <= most))
            return BDSSM_ERR_UNSUPPORTED;
        const double x = static_cast<double>(scale) / s->cap;
        g.two_x_log2 = static_cast<float>(2 * x * log2e);
        g.half_cap = static_cast<float>(0.5 / x);
        // tanh(x) = x (c0 + c1 x^2 + c2 x^4 + c3 x^6) up to 1/2, in powers of two of the raw score. Its
        // terms stay ordinary numbers for any x from 2^-12 to 2^12 per score
        const double c[4] = {0.999999456, -0.333263179, 0.131902966, -0.0444022263};
        double power = s->cap * log2e * x;
        for (int i = 0; i < 4; ++i, power *= x * x)
            g.q[i] = static_cast<float>(c[i] * power);
        g.fast = bf16 && s->cap <= 256.f && x >= 0x1p-12 && x <= 0x1p12;
    }
    g.slopes = s->slopes, g.prefix = s->prefix, g.first = s->first, g.last = s->last;
    r[0] = rng(s->slopes, a->H * 4ll);
    r[1] = rng(s->prefix, a->batch * 4ll);
    r[2] = rng(s->first, a->tokens * 4);
    r[3] = rng(s->last, a->tokens * 4);
    return BDSSM_OK;
}

// Workspace of a step whose scoring is a.score.
size_t step_workspace(const bdssm_attn_dims *dims, int32_t block_len, int32_t max_len, const bdssm_attn_mask *mask, AttnArgs a)
{
    if (check_attn_dims(dims) != BDSSM_OK || check_attn_mask(mask) != BDSSM_OK || block_len < 0 || max_len < 0 ||
        static_cast<int64_t>(max_len) + block_len > kMaxPosition)
        return SIZE_MAX;
    if (dims->batch == 0 || block_len == 0)
        return 0;
    a.batch = dims->batch, a.H = dims->nheads, a.KV = dims->kv_heads;
    a.block_len = block_len, a.max_len = max_len;
    a.block = mask->block, a.window = mask->window, a.sinks = mask->sinks;
    if (!rows_fit(a))
        return SIZE_MAX;
    return attn_workspace(a, dims->headdim, dims->dtype == BDSSM_BF16);
}

bdssm_status attn_step(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk, const bdssm_kv_cache *cache,
                       const bdssm_attn_mask *mask, const bdssm_attn_scores *scores, bool scored, void *out, void *workspace,
                       size_t workspace_bytes, void *stream)
{
    AttnArgs a;
    AttnRanges r;
    Range more[4] = {};
    bdssm_status rc = prepare_attn(dims, chunk, cache, true, false, &a, &r);
    if (rc != BDSSM_OK)
        return rc;
    if ((rc = check_attn_mask(mask)) != BDSSM_OK)
        return rc;
    if (scored && (rc = prepare_scores(scores, mask->scale, dims->dtype == BDSSM_BF16, &a, more)) != BDSSM_OK)
        return rc;
    if (!out && a.tokens > 0)
        return BDSSM_ERR_NULL;
    if (!aligned(out) || !aligned(workspace))
        return BDSSM_ERR_ALIGN;
    const Range ro = rng(out, a.tokens * a.H * dims->headdim * elt(dims->dtype));
    const Range in[] = {r.q, r.k, r.v, r.kp, r.vp, r.table, r.lens, r.starts, more[0], more[1], more[2], more[3]};
    for (Range q : in)
        if (overlap(ro, q))
            return BDSSM_ERR_ALIAS;
    if (a.batch == 0 || a.block_len == 0 || a.tokens == 0)
        return BDSSM_OK;
    a.scale = mask->scale, a.block = mask->block, a.window = mask->window, a.sinks = mask->sinks;
    a.by_block = Divisor(mask->block > 0 ? mask->block : 1);
    a.by_group = Divisor(dims->nheads / dims->kv_heads);
    a.out = out;
    if (!rows_fit(a))
        return BDSSM_ERR_UNSUPPORTED;
    const bool bf16 = dims->dtype == BDSSM_BF16;
    const AttnPlan p = attn_plan(a, dims->headdim, bf16);
    if (p.groups > kMaxGroups)
        return BDSSM_ERR_UNSUPPORTED;
    if (p.ws_bytes > 0) {
        if (!workspace || workspace_bytes < p.ws_bytes)
            return BDSSM_ERR_WORKSPACE;
        const Range rw = rng(workspace, static_cast<int64_t>(p.ws_bytes));
        for (Range q : in)
            if (overlap(rw, q))
                return BDSSM_ERR_ALIAS;
        if (overlap(rw, ro))
            return BDSSM_ERR_ALIAS;
    }
    const auto launch = !scored ? launch_attn : a.score.cap_log2 == 0.f ? launch_attn_ranged
                        : a.score.fast          ? launch_attn_capped
                                                : launch_attn_exact;
    return launched(launch(a, dims->headdim, bf16, p, workspace, static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace bdssm

using namespace bdssm;

extern "C" size_t bdssm_attn_step_workspace(const bdssm_attn_dims *dims, int32_t block_len, int32_t max_len,
                                            const bdssm_attn_mask *mask)
{
    return step_workspace(dims, block_len, max_len, mask, AttnArgs{});
}

extern "C" size_t bdssm_attn_step_ex_workspace(const bdssm_attn_dims *dims, int32_t block_len, int32_t max_len,
                                               const bdssm_attn_mask *mask, const bdssm_attn_scores *scores)
{
    AttnArgs a{};
    Range r[4];
    if (check_attn_dims(dims) != BDSSM_OK || check_attn_mask(mask) != BDSSM_OK ||
        prepare_scores(scores, mask->scale, dims->dtype == BDSSM_BF16, &a, r) != BDSSM_OK)
        return SIZE_MAX;
    return step_workspace(dims, block_len, max_len, mask, a);
}

extern "C" bdssm_status bdssm_attn_step(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk,
                                        const bdssm_kv_cache *cache, const bdssm_attn_mask *mask, void *out,
                                        void *workspace, size_t workspace_bytes, void *stream)
{
    return attn_step(dims, chunk, cache, mask, nullptr, false, out, workspace, workspace_bytes, stream);
}

extern "C" bdssm_status bdssm_attn_step_ex(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk,
                                           const bdssm_kv_cache *cache, const bdssm_attn_mask *mask,
                                           const bdssm_attn_scores *scores, void *out, void *workspace,
                                           size_t workspace_bytes, void *stream)
{
    return attn_step(dims, chunk, cache, mask, scores, true, out, workspace, workspace_bytes, stream);
}

extern "C" bdssm_status bdssm_kv_append(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk,
                                        const bdssm_kv_cache *cache, int32_t *lens_out, void *stream)
{
    AttnArgs a;
    AttnRanges r;
    bdssm_status rc = prepare_attn(dims, chunk, cache, false, true, &a, &r);
    if (rc != BDSSM_OK)
        return rc;
    if (!aligned4(lens_out))
        return BDSSM_ERR_ALIGN;
    const Range rl = rng(lens_out, a.batch * 4ll);
    for (Range w : {r.kp, r.vp, rl})
        for (Range q : {r.k, r.v, r.table, r.lens, r.starts})
            if (overlap(w, q))
                return BDSSM_ERR_ALIAS;
    if (overlap(r.kp, r.vp) || overlap(rl, r.kp) || overlap(rl, r.vp))
        return BDSSM_ERR_ALIAS;
    if (a.batch == 0)
        return BDSSM_OK;
    const int per16 = 16 / elt(dims->dtype);
    const int head_pieces = dims->headdim / per16, row_pieces = dims->kv_heads * head_pieces;
    const int64_t units = a.tokens > 0 ? static_cast<int64_t>(a.block_len) * row_pieces : 0;
    const int64_t blocks = units > 0 ? (units + 255) / 256 : 1;  // one is left to write lens_out
    if (blocks > (1 << 23))  // threads along x have to fit 32 bits
        return BDSSM_ERR_UNSUPPORTED;
    k_append<<<dim3(static_cast<unsigned>(blocks), a.batch), 256, 0, static_cast<hipStream_t>(stream)>>>(
        a, lens_out, head_pieces, row_pieces, per16);
    return launched(hipGetLastError());
}
