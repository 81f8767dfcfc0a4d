// Rotary positions of queries and keys (bdssm_rotary_step), the same on the way into the pages
// (bdssm_rotary_append), and the table of frequencies (bdssm_rotary_turns).
#include <algorithm>
#include <cmath>

#include "attn.h"
#include "internal.h"

namespace bdssm {
namespace {

// How the channels of a rotated head are split over threads; a unit is what one thread takes:
enum Layout {
    kPairsInPiece,  // interleaved: a 16-byte piece, which holds whole pairs
    kTwoPieces,     // halves of whole pieces: the two pieces of E pairs, or a piece past dim
    kSingle         // halves that end inside a piece: one pair, or one channel past dim
};

struct RotaryArgs {
    AttnArgs a;  // the chunk, and the cache where keys go into it
    void *qo, *ko;
    int64_t qo_stride, ko_stride;
    const uint64_t *turns;
    const int *positions;
    int *lens_out;
    float scale;
    int dim, headdim, tok;  // tok: tokens of a workgroup
    int q_heads;            // 0 without queries
    int units;              // of a rotated head
    int rotated;            // units of a token's rotated heads; its values' pieces come after them
    Divisor by_pairs, by_unit, by_token;
};

// cos and sin of 2 pi t / 2^64: the quarter turn nearest to t, and of what is left, pi / 4 at most,
// the series (the next terms are 2e-9 of the sine and 1e-10).
__device__ __forceinline__ float2 cos_sin(uint64_t t)
{
    const uint64_t quarter = (t + (uint64_t{1} << 61)) >> 62;
    // what is left is below 2^61 in magnitude: two bits up, and the upper word of it
    const int rest = static_cast<int>(static_cast<int64_t>((t - (quarter << 62)) << 2) >> 32);
    const float x = static_cast<float>(rest) * static_cast<float>(6.283185307179586476925 * 0x1p-34), u = x * x;
    float s = 1.f / 362880.f, c = -1.f / 3628800.f;
    s = fmaf(s, u, -1.f / 5040.f);
    s = fmaf(s, u, 1.f / 120.f);
    s = fmaf(s, u, -1.f / 6.f);
    s = fmaf(s * u, x, x);
    c = fmaf(c, u, 1.f / 40320.f);
    c = fmaf(c, u, -1.f / 720.f);
    c = fmaf(c, u, 1.f / 24.f);
    c = fmaf(c, u, -0.5f);
    c = fmaf(c, u, 1.f);
    const bool odd = quarter & 1;
    const float cs = odd ? s : c, sn = odd ? c : s;
    return make_float2((quarter + 1) & 2 ? -cs : cs, quarter & 2 ? -sn : sn);
}

template <typename T>
struct alignas(16) Piece {
    T v[16 / sizeof(T)];
};

template <typename T>
__device__ __forceinline__ void turn_pair(T &a, T &b, float2 t)
{
    const float x = static_cast<float>(a), y = static_cast<float>(b);
    a = static_cast<T>(fmaf(x, t.x, -(y * t.y)));
    b = static_cast<T>(fmaf(x, t.y, y * t.x));
}

// A workgroup takes `tok` tokens of one stream. The scaled cosines and sines of their pairs are
// made once, in LDS, for all heads; the threads walk the units of (token, head): queries, keys,
// values. Bound by the rows' bytes: a step of 34,000 tokens of 20 + 4 heads x 128 takes 62 us, 6.8
// TB/s both ways (a large copy by the library: 4.9), with values and into pages 75 us, 6.5. What that
// took: four pieces of a thread in flight (two: 122 us), 4 tokens a workgroup (16, whose first loads
// nothing covers: 112 us; eight pieces in flight no better), and, where the outputs are more than the
// L2s hold, stores that do not stay in them (STREAM; 101 us without). One block of 32: 2.9 us, the
// launch and the way to the stream's length. Halves that end inside a piece go a pair a thread, 2.4
// TB/s.
template <typename T, int LAYOUT, bool APPEND, bool STREAM>
__global__ __launch_bounds__(256) void k_rotary(RotaryArgs r)
{
    constexpr int E = 16 / sizeof(T);
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const AttnArgs &a = r.a;
    const int b = blockIdx.y, pairs = r.dim / 2;
    float2 *turn = reinterpret_cast<float2 *>(lds);                          // [tok][pairs]
    int64_t *slots = reinterpret_cast<int64_t *>(lds) + r.tok * pairs;       // [tok]: offset in a pool, head 0; -1: none
    const AttnStream s = attn_rows(a, b, a.lens ? a.lens[b] : 0);
    const int64_t held = static_cast<int64_t>(a.max_pages) << a.page_shift;
    if (APPEND && r.lens_out && blockIdx.x == 0 && threadIdx.x == 0) {
        const int64_t end = static_cast<int64_t>(s.len) + s.n;
        r.lens_out[b] = static_cast<int>(end < held ? end : held);
    }
    const int i0 = blockIdx.x * r.tok, n = s.n - i0 < r.tok ? s.n - i0 : r.tok;
    if (n <= 0)
        return;
    const int per_token = static_cast<int>(r.by_token.d), total = n * per_token, page = 1 << a.page_shift;

    struct Unit {
        int i, head, u;  // token of the workgroup; q heads, then KV (keys), then KV (values); unit of the head
    };
    auto unit = [&](int x) {
        const int i = r.by_token(x), y = x - i * per_token;
        if (APPEND && y >= r.rotated) {
            const int per = r.headdim / E;  // a power of two
            const int h = (y - r.rotated) / per;
            return Unit{i, r.q_heads + a.KV + h, y - r.rotated - h * per};
        }
        const int h = r.by_unit(y);
        return Unit{i, h, y - h * r.units};
    };
    auto row = [&](const Unit &x, const void *q, int64_t qs, const void *k, int64_t ks) {  // of a rotated head
        const int64_t at = s.row0 + i0 + x.i;
        return x.head < r.q_heads
                   ? const_cast<T *>(static_cast<const T *>(q)) + at * qs + static_cast<int64_t>(x.head) * r.headdim
                   : const_cast<T *>(static_cast<const T *>(k)) + at * ks + static_cast<int64_t>(x.head - r.q_heads) * r.headdim;
    };
    // a unit's channels: `first` (a piece, or one channel) and, where it is a pair's, `second`
    auto first_of = [&](const Unit &x) {
        if (LAYOUT == kPairsInPiece)
            return x.u * E;
        if (LAYOUT == kTwoPieces)
            return x.u * E < pairs ? x.u * E : x.u * E + pairs;
        return x.u < pairs ? x.u : x.u + pairs;
    };
    auto is_pair = [&](const Unit &x) { return LAYOUT == kTwoPieces ? x.u * E < pairs : LAYOUT == kSingle && x.u < pairs; };
    struct Data {
        Piece<T> a, b;
    };
    auto load = [&](const Unit &x) {
        Data d;
        if (APPEND && x.head >= r.q_heads + a.KV) {
            d.a = *reinterpret_cast<const Piece<T> *>(static_cast<const T *>(a.v) + (s.row0 + i0 + x.i) * a.v_stride +
                                                      static_cast<int64_t>(x.head - r.q_heads - a.KV) * r.headdim + x.u * E);
            return d;
        }
        const T *from = row(x, a.q, a.q_stride, a.k, a.k_stride) + first_of(x);
        if constexpr (LAYOUT == kSingle) {
            d.a.v[0] = from[0];
            if (is_pair(x))
                d.b.v[0] = from[pairs];
        } else {
            d.a = *reinterpret_cast<const Piece<T> *>(from);
            if (is_pair(x))
                d.b = *reinterpret_cast<const Piece<T> *>(from + pairs);
        }
        return d;
    };
    auto put = [](T *to, const Piece<T> &p) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        if constexpr (STREAM)
            __builtin_nontemporal_store(__builtin_bit_cast(u32x4, p), reinterpret_cast<u32x4 *>(to));
        else
            *reinterpret_cast<Piece<T> *>(to) = p;
    };
    auto store_at = [&](T *to, const Unit &x, const Data &d) {
        if constexpr (LAYOUT == kSingle) {
            to[0] = d.a.v[0];
            if (is_pair(x))
                to[pairs] = d.b.v[0];
        } else {
            put(to, d.a);
            if (is_pair(x))
                put(to + pairs, d.b);
        }
    };
    auto store = [&](const Unit &x, Data d) {
        if (APPEND && x.head >= r.q_heads + a.KV) {
            if (slots[x.i] >= 0)
                put(static_cast<T *>(a.vp) + slots[x.i] +
                        static_cast<int64_t>(x.head - r.q_heads - a.KV) * page * r.headdim + x.u * E,
                    d.a);
            return;
        }
        const float2 *t = turn + x.i * pairs;
        const int c = first_of(x);
        if constexpr (LAYOUT == kPairsInPiece) {
#pragma unroll
            for (int e = 0; e < E; e += 2)
                if (c + e < r.dim)
                    turn_pair(d.a.v[e], d.a.v[e + 1], t[(c + e) / 2]);
        } else if (is_pair(x)) {
#pragma unroll
            for (int e = 0; e < (LAYOUT == kSingle ? 1 : E); ++e)
                turn_pair(d.a.v[e], d.b.v[e], t[c + e]);
        }
        if (x.head < r.q_heads || r.ko)
            store_at(row(x, r.qo, r.qo_stride, r.ko, r.ko_stride) + c, x, d);
        if (APPEND && x.head >= r.q_heads && slots[x.i] >= 0)
            store_at(static_cast<T *>(a.kp) + slots[x.i] + static_cast<int64_t>(x.head - r.q_heads) * page * r.headdim + c, x, d);
    };

    // U units of a thread are loaded before the first of them is stored, the first U before the cosines
    // are made
    constexpr int U = LAYOUT == kTwoPieces ? 2 : 4;
    Data d[U];
    auto load_from = [&](int x0) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int x = x0 + 256 * k;
            d[k] = load(unit(x < total ? x : total - 1));
        }
    };
    load_from(threadIdx.x);
    for (int y = threadIdx.x; y < n * pairs; y += 256) {
        const int i = r.by_pairs(y), f = y - i * pairs;
        const int64_t p = r.positions ? r.positions[s.row0 + i0 + i] : static_cast<int64_t>(s.len) + i0 + i;
        const float2 t = cos_sin(static_cast<uint64_t>(p) * r.turns[f]);
        turn[y] = make_float2(t.x * r.scale, t.y * r.scale);
    }
    if (APPEND && threadIdx.x < n) {
        const int64_t j = static_cast<int64_t>(s.len) + i0 + threadIdx.x;
        const int pg = j < held ? a.table[static_cast<int64_t>(b) * a.max_pages + (j >> a.page_shift)] : -1;
        slots[threadIdx.x] = pg < 0 || pg >= a.num_pages
                                 ? -1
                                 : (static_cast<int64_t>(pg) * a.KV * page + (j & (page - 1))) * r.headdim;
    }
    __syncthreads();
    for (int x0 = threadIdx.x; x0 < total; x0 += 256 * U) {
        if (x0 != static_cast<int>(threadIdx.x))
            load_from(x0);
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (x0 + 256 * k < total)
                store(unit(x0 + 256 * k), d[k]);
    }
}

template <typename T, bool APPEND, bool STREAM>
void launch(const RotaryArgs &r, Layout layout, dim3 grid, size_t lds, hipStream_t st)
{
    if (layout == kPairsInPiece)
        k_rotary<T, kPairsInPiece, APPEND, STREAM><<<grid, 256, lds, st>>>(r);
    else if (layout == kTwoPieces)
        k_rotary<T, kTwoPieces, APPEND, STREAM><<<grid, 256, lds, st>>>(r);
    else
        k_rotary<T, kSingle, APPEND, false><<<grid, 256, lds, st>>>(r);
}

template <typename T, bool APPEND>
void launch(const RotaryArgs &r, Layout layout, dim3 grid, size_t lds, bool stream, hipStream_t st)
{
    if (stream)
        launch<T, APPEND, true>(r, layout, grid, lds, st);
    else
        launch<T, APPEND, false>(r, layout, grid, lds, st);
}

// Rows of a tensor, in bytes.
struct Rows {
    const void *p;
    int64_t stride, width, n;
    Range span() const { return rng(p, n > 0 ? (n - 1) * stride + width : 0); }
    bool same(const Rows &o) const { return p == o.p && width == o.width && (stride == o.stride || n <= 1); }
};

// Whether rows share memory. Rows of one stride that keep apart within it do not, though their spans
// do: slices of one projection.
bool overlap(const Rows &x, const Rows &y)
{
    if (!overlap(x.span(), y.span()))
        return false;
    if (x.stride != y.stride)
        return true;
    int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(y.p) - reinterpret_cast<uintptr_t>(x.p)) % x.stride;
    d = d < 0 ? d + x.stride : d;
    return d < x.width || d + y.width > x.stride;
}

bdssm_status check_rotary(const bdssm_rotary *ro, int headdim)
{
    if (!ro)
        return BDSSM_ERR_NULL;
    if (ro->dim < 2 || ro->dim % 2 != 0 || ro->dim > headdim)
        return BDSSM_ERR_SHAPE;
    if ((ro->interleaved != 0 && ro->interleaved != 1) || ro->scale - ro->scale != 0.f)
        return BDSSM_ERR_UNSUPPORTED;
    if (!ro->turns)
        return BDSSM_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(ro->turns) & 7u) != 0 || !aligned4(ro->positions))
        return BDSSM_ERR_ALIGN;
    return BDSSM_OK;
}

// Both calls, once their chunk (and cache) is checked: outputs, overlaps, launch.
bdssm_status run(const bdssm_attn_dims *d, const AttnArgs &a, const AttnRanges &in, const bdssm_rotary *ro,
                 const bdssm_rotary_out *out, bool append, int32_t *lens_out, hipStream_t st)
{
    const int e = elt(d->dtype), per16 = 16 / e;
    const int64_t qw = static_cast<int64_t>(d->nheads) * d->headdim, kw = static_cast<int64_t>(d->kv_heads) * d->headdim;
    const bdssm_rotary_out none{};
    const bdssm_rotary_out &o = out ? *out : none;
    if (a.tokens > 0 && ((a.q != nullptr) != (o.q != nullptr) || (append ? o.k && !a.k : (a.k != nullptr) != (o.k != nullptr)) ||
                         (!a.q && !a.k)))
        return BDSSM_ERR_NULL;
    if ((o.q && o.q_stride < qw) || (o.k && o.k_stride < kw))
        return BDSSM_ERR_SHAPE;
    if ((o.q && o.q_stride > kMaxStride) || (o.k && o.k_stride > kMaxStride))
        return BDSSM_ERR_UNSUPPORTED;
    if (!aligned(o.q) || !aligned(o.k) || (o.q && o.q_stride % per16 != 0) || (o.k && o.k_stride % per16 != 0) ||
        !aligned4(lens_out))
        return BDSSM_ERR_ALIGN;
    auto rows = [&](const void *p, int64_t stride, int64_t width) { return Rows{p, stride * e, width * e, a.tokens}; };
    const Rows q = rows(a.q, a.q_stride, qw), k = rows(a.k, a.k_stride, kw), v = rows(append ? a.v : nullptr, a.v_stride, kw);
    const Rows qo = rows(o.q, o.q_stride, qw), ko = rows(o.k, o.k_stride, kw);
    const Range turns = rng(ro->turns, ro->dim / 2 * 8), at = rng(ro->positions, a.tokens * 4), rl = rng(lens_out, a.batch * 4ll);
    // in place, or apart from everything
    if ((!qo.same(q) && overlap(qo, q)) || (!ko.same(k) && overlap(ko, k)) || overlap(qo, k) || overlap(ko, q) ||
        overlap(qo, v) || overlap(ko, v) || overlap(qo, ko))
        return BDSSM_ERR_ALIAS;
    for (const Rows &w : {qo, ko})
        for (Range x : {in.kp, in.vp, in.table, in.lens, in.starts, turns, at, rl})
            if (overlap(w.span(), x))
                return BDSSM_ERR_ALIAS;
    for (Range w : {in.kp, in.vp, rl})
        for (Range x : {q.span(), k.span(), v.span(), in.table, in.lens, in.starts, turns, at})
            if (overlap(w, x))
                return BDSSM_ERR_ALIAS;
    if (overlap(in.kp, in.vp) || overlap(rl, in.kp) || overlap(rl, in.vp))
        return BDSSM_ERR_ALIAS;
    const int64_t most = std::min<int64_t>(a.block_len, a.tokens);  // tokens of a stream
    if (most > 1 << 24)  // threads along x have to fit 32 bits; there a workgroup has two tokens at least
        return BDSSM_ERR_UNSUPPORTED;
    if (a.batch == 0 || (!append && (a.tokens == 0 || a.block_len == 0)))
        return BDSSM_OK;
    RotaryArgs r{};
    r.a = a;
    r.qo = o.q, r.ko = o.k, r.qo_stride = o.q_stride, r.ko_stride = o.k_stride;
    r.turns = ro->turns, r.positions = ro->positions, r.lens_out = lens_out;
    r.scale = ro->scale, r.dim = ro->dim, r.headdim = d->headdim;
    r.q_heads = a.q ? d->nheads : 0;
    const int pairs = ro->dim / 2;
    const Layout layout = ro->interleaved ? kPairsInPiece : pairs % per16 == 0 ? kTwoPieces : kSingle;
    r.units = layout == kPairsInPiece ? d->headdim / per16 : layout == kTwoPieces ? (d->headdim - pairs) / per16 : d->headdim - pairs;
    r.rotated = (r.q_heads + (a.k ? d->kv_heads : 0)) * r.units;
    r.tok = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(layout == kTwoPieces ? 2 : 4, a.tokens / 2048)));
    r.by_pairs = Divisor(pairs), r.by_unit = Divisor(r.units);
    r.by_token = Divisor(r.rotated + (append ? d->kv_heads * d->headdim / per16 : 0));
    const int64_t blocks = std::max<int64_t>(1, (most + r.tok - 1) / r.tok);  // one is left to write lens_out
    const dim3 grid(static_cast<unsigned>(blocks), a.batch);
    const size_t lds = static_cast<size_t>(r.tok) * (pairs + 1) * 8;
    // the eight L2s hold 32 MB
    const bool stream = a.tokens * ((r.q_heads ? qw : 0) + (a.k ? kw : 0)) * e > 32 << 20;
    if (d->dtype == BDSSM_BF16)
        append ? launch<__bf16, true>(r, layout, grid, lds, stream, st) : launch<__bf16, false>(r, layout, grid, lds, stream, st);
    else
        append ? launch<float, true>(r, layout, grid, lds, stream, st) : launch<float, false>(r, layout, grid, lds, stream, st);
    return launched(hipGetLastError());
}

}  // namespace
}  // namespace bdssm

using namespace bdssm;

extern "C" bdssm_status bdssm_rotary_turns(const bdssm_rotary_freqs *f, uint64_t *turns)
{
    if (!f || !turns)
        return BDSSM_ERR_NULL;
    if (f->dim < 2 || f->dim % 2 != 0 || f->dim > 512)
        return BDSSM_ERR_SHAPE;
    const bool plain = f->kind == BDSSM_ROTARY_PLAIN, parts = f->kind == BDSSM_ROTARY_PARTS;
    if (f->kind < BDSSM_ROTARY_PLAIN || f->kind > BDSSM_ROTARY_PARTS || !(f->base >= 1.) || !std::isfinite(f->base) ||
        (!plain && (!(f->factor > 0.) || !std::isfinite(f->factor))) || (f->kind == BDSSM_ROTARY_BASE && f->dim == 2) ||
        (parts && (f->trained < 1 || !(f->low < f->high) || !std::isfinite(f->low) || !std::isfinite(f->high))))
        return BDSSM_ERR_UNSUPPORTED;
    // in 64 bits of fraction (x86's long double): turns per position are right to 2^-64 or so of
    // themselves, and of a turn
    const long double two_pi = 6.283185307179586476925286766559L, dim = f->dim;
    long double base = f->base;
    if (f->kind == BDSSM_ROTARY_BASE)
        base *= powl(f->factor, dim / (dim - 2));
    for (int i = 0; i < f->dim / 2; ++i) {
        long double per = powl(base, -2 * i / dim);  // radians
        if (f->kind == BDSSM_ROTARY_LINEAR)
            per /= f->factor;
        if (parts) {
            long double g = (f->trained * per / two_pi - f->low) / (static_cast<long double>(f->high) - f->low);
            g = g < 0 ? 0 : g > 1 ? 1 : g;
            per *= g + (1 - g) / f->factor;
        }
        per /= two_pi;
        // whole turns, which a factor far below 1 makes, count for nothing
        const long double x = roundl((per - floorl(per)) * 0x1p64L);
        turns[i] = x >= 0x1p64L ? 0 : static_cast<uint64_t>(x);
    }
    return BDSSM_OK;
}

extern "C" bdssm_status bdssm_rotary_step(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk,
                                          const bdssm_rotary *rotary, const int32_t *lens, const bdssm_rotary_out *out,
                                          void *stream)
{
    bdssm_status rc = check_attn_dims(dims);
    if (rc != BDSSM_OK)
        return rc;
    if (!chunk || !out)
        return BDSSM_ERR_NULL;
    if ((rc = check_rotary(rotary, dims->headdim)) != BDSSM_OK)
        return rc;
    if (chunk->block_len < 0 || chunk->tokens < 0 ||
        (!chunk->starts && chunk->tokens != static_cast<int64_t>(dims->batch) * chunk->block_len))
        return BDSSM_ERR_SHAPE;
    if (chunk->tokens > INT_MAX || (chunk->q && chunk->q_stride > kMaxStride) || (chunk->k && chunk->k_stride > kMaxStride))
        return BDSSM_ERR_UNSUPPORTED;
    const int e = elt(dims->dtype), per16 = 16 / e;
    if ((chunk->q && chunk->q_stride < static_cast<int64_t>(dims->nheads) * dims->headdim) ||
        (chunk->k && chunk->k_stride < static_cast<int64_t>(dims->kv_heads) * dims->headdim))
        return BDSSM_ERR_SHAPE;
    if (!aligned(chunk->q) || !aligned(chunk->k) || !aligned4(chunk->starts) || !aligned4(lens) ||
        (chunk->q && chunk->q_stride % per16 != 0) || (chunk->k && chunk->k_stride % per16 != 0))
        return BDSSM_ERR_ALIGN;
    AttnArgs a{};
    a.q = chunk->q, a.k = chunk->k;
    a.q_stride = chunk->q_stride, a.k_stride = chunk->k_stride;
    a.tokens = chunk->tokens, a.starts = chunk->starts, a.block_len = chunk->block_len;
    a.lens = rotary->positions ? nullptr : lens;
    a.max_len = INT_MAX;
    a.batch = dims->batch, a.H = dims->nheads, a.KV = dims->kv_heads;
    AttnRanges in{};
    in.lens = rng(a.lens, dims->batch * 4ll);
    in.starts = rng(chunk->starts, dims->batch > 0 ? (dims->batch + 1) * 4ll : 0);
    return run(dims, a, in, rotary, out, false, nullptr, static_cast<hipStream_t>(stream));
}

extern "C" bdssm_status bdssm_rotary_append(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk,
                                            const bdssm_kv_cache *cache, const bdssm_rotary *rotary,
                                            const bdssm_rotary_out *out, int32_t *lens_out, void *stream)
{
    AttnArgs a;
    AttnRanges in;
    bdssm_status rc = prepare_attn(dims, chunk, cache, chunk && chunk->q, true, &a, &in);
    if (rc != BDSSM_OK)
        return rc;
    if ((rc = check_rotary(rotary, dims->headdim)) != BDSSM_OK)
        return rc;
    return run(dims, a, in, rotary, out, true, lens_out, static_cast<hipStream_t>(stream));
}
