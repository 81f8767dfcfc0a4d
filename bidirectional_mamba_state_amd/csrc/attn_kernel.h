// Attention of a chunk over a paged cache on the matrix cores (gfx950): one pass over the keys
// with a running softmax, for both element types.
//
// Work split. The query heads of one KV head are packed with the tokens into rows, row
// r = token * G + head-in-group, so that a tile of keys and values is read once for all of
// them. A workgroup owns one (stream, KV head), a tile of RT = 32 WM rows and a range of the
// keys that those rows attend to; a wavefront owns 32 rows and, where few rows leave
// wavefronts free (WK > 1), every WK-th part of each key tile. A long cache is cut into
// `nsplit` ranges; partial results (unnormalized rows, maximum, sum) are joined by k_attn_join.
//
// Products. S^T = K Q^T and O^T = V^T P^T, with keys (then channels) along the rows of the
// 32 x 32 accumulators and queries along their columns: a lane holds scores of one query only,
// so the softmax's maximum and sum need one exchange (between the two halves of a wavefront),
// its rescaling none, and the accumulators of S^T are the B operand of the second product as
// they stand. Their row order, lane half hf and register i <-> key 8 (i/4) + 4 hf + i%4, is met
// by reading V in that order.
//
// Softmax. Scores are scaled to powers of two (scale log2 e folded into one fma before exp2).
// The reference m of a query is set 8 above the maximum, and raised, with its sums rescaled, only
// when a tile's maximum exceeds it: weights are 1 at most (a sum overflows only where the values'
// own would), and the largest is 2^-8 at least, which float32 sums and bf16 weights hold as well.
// With bf16 values each weight is rounded to bf16: the matrix cores take both factors in one type,
// and float32 products run at an eighth of the rate. Their sum is of the rounded weights, so that
// the weights that are used add up to one exactly; it is float32, as are maxima and weighted sums.
//
// Copies. Keys and values go from the pages (or the chunk's rows) straight into LDS, 1 KB a
// copy, each copy inside one page (a page holds 16 tokens or more, a copy 8 at most); the
// 16-byte pieces of a row are permuted on the way (swz_k, swz_v) so that the operand reads are
// free of bank conflicts. Two stages: the next tile is in flight while one is computed.
//
// Masks. Per tile a 64-bit mask says which keys exist, are held and are attended to by any row
// of the workgroup; the values of the others (which may hold anything, NaN included) are cleared
// in LDS before use. Scores are selected per element in tiles that some row of a wavefront does
// not see whole; the other tiles skip that. Values of keys that only some rows attend to may hold
// infinities and NaN too: see repair.
//
// What bounds it, measured (a large bf16 matrix product reaches 1,258 TFLOP/s here, float32 153, a
// large copy 4.9 TB/s both ways):
//  - single tokens: HBM reads, 5.7 TB/s (64 streams x 32,768 tokens, 6 heads a group: 370 us);
//  - a block of 32 on 262,144 tokens, 5 heads a group of 64: HBM and the vector unit together,
//    3.7 TB/s at 590 TFLOP/s (146 us with its join of 8 us);
//  - many rows, headdim 128: the matrix cores (42 % busy) share the clock with the exponentials
//    (34 %) and with LDS, whose operand reads take half as long as the products; 970 TFLOP/s
//    (a prompt chunk of 8,192 on 8,192, 20 heads: 1.06 ms);
//  - many rows, headdim 64: no unit alone (vector 54 % busy, half of it exponentials, matrix cores
//    37 %, so that they take turns more than they overlap); copies and the wait for them before
//    every tile are a quarter (1,323 us with them, 1,006 without); 880 TFLOP/s on equal streams,
//    740 on unequal ones (64 x 16-32K tokens, 768 rows: 1.23 ms), where short row tiles leave
//    wavefronts idle;
//  - float32: the matrix cores, 100 to 125 TFLOP/s;
//  - a cap: the vector unit beside them (48 % busy, matrix cores 34 %): the prompt chunk 1.30 ms, the
//    unequal streams 1.84; a bias: the prompt chunk 1.23 ms, the unequal streams 1.37, where the vector
//    unit is 68 % busy; both: 1.70 and 2.12 ms. At headdim 64 these kernels spill 7 (bias) and 8 (cap)
//    of their 128 registers, the plain one none;
//  - documents packed into a prompt (8,191 tokens in some of 700, 16 heads over 4): neither unit (vector
//    46 and 36 % busy, matrix cores 18 and 24 % at headdim 64 and 128; waits 38 and 35 %): a workgroup
//    walks seven tiles on average, behind its start; 41 and 60 us, 5.7 of them the order of row tiles.
//    As streams of their own they take 34 and 52 us (documents of 60 to 2,000: packed 0.7 to 1.3 times
//    that).
// Eight wavefronts of 32 rows, four a SIMD at headdim 64, did better than four of 64 (half the
// LDS reads, but nothing hides a wavefront's own exponentials: 1340 against 1020 us on the
// prompt), than a third stage, 128-key tiles or a scheduled overlap inside a wavefront (no
// difference, or registers spilled).
#pragma once

#include <limits.h>

#include <type_traits>

#include "attn.h"
#include "internal.h"
#include "mfma_tiles.h"
#include "wave_ops.h"

namespace bdssm {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kAbove = 8.f;  // see "Softmax" above

template <typename T, int D>
struct Tile;

template <int D>
struct Tile<__bf16, D> {
    typedef bf16x8 Frag;
    static constexpr int ROWB = 2 * D, STEPS = D / 16;
    // a K operand read takes one piece of 16 consecutive rows (and of 16 more), a V operand
    // read (transposing) four pieces of 4 consecutive rows: distinct bank groups for each
    static __device__ __forceinline__ int swz_k(int r) { return D == 128 ? r & 15 : (r >> 1) & 7; }
    static __device__ __forceinline__ int swz_v(int r) { return D == 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2; }
    static __device__ __forceinline__ f32x16 qk(Frag k, Frag q, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q, c, 0, 0, 0);
    }
};

template <int D>
struct Tile<float, D> {
    typedef f32x4 Frag;
    static constexpr int ROWB = 4 * D, STEPS = D / 8;
    static __device__ __forceinline__ int swz_k(int r) { return r & 15; }
    static __device__ __forceinline__ int swz_v(int) { return 0; }  // read by 128-byte runs of a row
    static __device__ __forceinline__ f32x16 qk(Frag k, Frag q, f32x16 c)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(k[e], q[e], c, 0, 0, 0);
        return c;
    }
};

// the larger of a lane's value and its counterpart's in the other half of the wavefront
__device__ __forceinline__ float half_max(float v)
{
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float half_sum(float v)
{
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// s plus weights 2e and 2e + 1 of w
__device__ __forceinline__ float add_pair(bf16x8 w, int e, float s)
{
    const bf16x2 ones = {static_cast<__bf16>(1.f), static_cast<__bf16>(1.f)};
    return __builtin_amdgcn_fdot2_f32_bf16(bf16x2{w[2 * e], w[2 * e + 1]}, ones, s, false);
}

// the n lowest bits, for any n
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

template <int N>
struct Int {
    static constexpr int value = N;
};

// whether any lane of a workgroup of NW wavefronts found something
template <int NW>
__device__ __forceinline__ bool anyone(int *found, bool mine)
{
    const int any_mine = __ballot(mine) != 0;
    if ((threadIdx.x & 63) == 0)
        found[threadIdx.x >> 6] = any_mine;
    __syncthreads();
    int any = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i)
        any |= found[i];
    return __builtin_amdgcn_readfirstlane(any) != 0;
}

// A workgroup's rows and tiles of keys, as k_attn has them.
struct RowRange {
    int b, kvh, split, nsplit, r_first, r_end, t0, t1, ns, nw, w0, c0, tk, nwaves;
};
// The same with the least and the most of what its rows attend to (see Sight).
struct Bounds {
    int lo_min, lo_max, hi_min, hi_max, f_min, f_max;
};
struct RowRangeEx : RowRange {
    Bounds bounds;
};

// What a chunk token attends to: keys [lo, hi), and with a window the sinks in [first, hi).
struct Sight {
    int lo, hi, first;
};
constexpr int kNever = INT_MAX;  // lo and first of a token whose range leaves it nothing; its hi is 0

template <bool EX>
__device__ __forceinline__ Sight sight_of(const AttnArgs &a, const AttnStream &s, int end, int prefix, int tok)
{
    const int p = s.len + tok;
    Sight x = {a.window == 0 || p < a.window ? 0 : p - a.window + 1, end, 0};
    if (a.block != 0) {
        const int64_t h = static_cast<int64_t>(a.by_block(p) + 1) * a.block;
        x.hi = h < end ? static_cast<int>(h) : end;
    }
    if constexpr (EX) {
        auto within = [&](int v) { return v < 0 ? 0 : v > end ? end : v; };
        x.hi = x.hi > prefix ? x.hi : prefix;
        if (a.score.first) {
            x.first = within(a.score.first[s.row0 + tok]);
            x.lo = x.lo > x.first ? x.lo : x.first;
        }
        if (a.score.last) {
            const int last = within(a.score.last[s.row0 + tok]);
            x.hi = x.hi < last ? x.hi : last;
        }
        // without ranges the bounds are left to grow with the token, which the kernel relies on there
        if ((a.score.first || a.score.last) && x.lo >= x.hi && x.first >= (x.hi < a.sinks ? x.hi : a.sinks))
            x = {kNever, 0, kNever};
    }
    return x;
}

// positions below this are visible to a stream's every query, whatever the order
__device__ __forceinline__ int prefix_of(const AttnArgs &a, int b, int end)
{
    const int v = a.score.prefix ? a.score.prefix[b] : 0;
    return v < 0 ? 0 : v > end ? end : v;
}

// What a kernel does to scores and ranges beyond the mask of bdssm_attn_step: nothing; ranges of rows and
// a bias, each where it is given (AttnArgs::score); a cap, and those: as exactly as bf16 weights ask for
// (a cap of 256 or less, AttnScoring::fast), or as float32 can.
enum Mode { kPlain, kRanged, kCapped, kExact };

// Shaped scores, in powers of two.
//
// Cap: c tanh(x), x = s / c. Two forms: x Q(x^2), Q the polynomial with the least relative error up to
// some |x|; and 1 - 2 / (1 + e^2x), whose error is a few 2^-24 of c, and which an infinite score takes
// to +-1. Each costs: the polynomial a multiplication and an addition a term, the other two
// transcendentals, which take as long as eight additions.
//  - kExact: six terms up to 0.6 (5e-9), the other form from there on, where it is a few 2^-24 of the
//    score too; of both, where a wavefront's scores of a tile are not all small, the one that applies.
//  - kCapped: the other form (a few 2^-24 of c). At headdim 128, where a wavefront sees a whole tile and
//    all of its scores are below c / 2, four terms instead (5.4e-7 of the score: up to 1e-4 of a power
//    of two, a fortieth of the rounding of a bf16 weight), made along with the weights, where the
//    products hide them (a prompt of 8,192 on 8,192: 1.30 ms, 1.48 in the other form, 2.0 in front of
//    the weights). At 64 the 8 x 1 shape's registers are full (8 spilled, 36 bytes a lane): with both ways
//    more spills took what was saved.
//
// Constants are operands of the instructions themselves (add_mul): as values each took a vector
// register through the loop over tiles.
template <uint32_t BITS>
__device__ __forceinline__ float add_mul(float a, float b)  // a b + constant
{
    float r;
    asm("v_fmaak_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "n"(BITS));
    return r;
}
__device__ __forceinline__ float tanh_near(float x, float u)  // u = x^2, up to 0.36
{
    constexpr auto bits = [](float c) { return __builtin_bit_cast(uint32_t, c); };
    float t = u * -0.00585216868f + 0.020753629f;
    t = add_mul<bits(-0.0537687048f)>(t, u);
    t = add_mul<bits(0.13331689f)>(t, u);
    t = add_mul<bits(-0.333332833f)>(t, u);
    return fmaf(t * u, x, x);
}
__device__ __forceinline__ float capped_near(float s, const AttnScoring &g)
{
    const float x = s * g.x_per_score;
    return g.cap_log2 * tanh_near(x, x * x);
}
__device__ __forceinline__ float capped(float s, const AttnScoring &g)
{
    const float x = s * g.x_per_score, u = x * x, t = tanh_near(x, u);
    float far = fmaf(-2.f, __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * (2.f * kLog2e))), 1.f);
    asm("" : "+v"(far));  // both, then one of the two: no branch around each score
    return g.cap_log2 * (u < 0.36f ? t : far);
}
// any scores, to a few 2^-24 of c
__device__ __forceinline__ float capped_any(float s, const AttnScoring &g)
{
    const float r = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(s * g.two_x_log2));
    return fmaf(r, -2.f * g.cap_log2, g.cap_log2);
}
// small scores: s times this
struct Poly {
    float q0, q1, q2, q3;
    __device__ __forceinline__ float operator()(float s) const
    {
        const float u = s * s;
        return fmaf(u, fmaf(u, fmaf(u, q3, q2), q1), q0);
    }
};

// Bias: a slope times the distance to the key. The softmax does not change when a row's scores
// move together, so the distance is taken from the nearest position that the row attends to
// (`from`): where a row sees only far keys, the common part, which float32 would round, is left out.
// A slope beyond 2^26 counts as 2^26: the nearest key then has all of the weight, unless scores differ by
// as much, and a slope times a distance (below 2^31), log2 e and the inverse of the scale (2^64 at most)
// stays finite. An infinity at the first key of a block, from which the others step, would reach the
// nearest. Where products start from the bias, one below -2^26 counts as that: weights are exp2 of one fma
// of the raw score, and the rounding of a reference of 2^26.6 leaves 4 in its exponent (kAbove is more); of
// one of 2^32, which a tile of far keys would set before the nearest comes, more than float32 holds.
constexpr float kSteepest = 0x1p26f;
__device__ __forceinline__ float slope_of(const AttnScoring &g, int head)
{
    const float s = g.slopes[head];
    return fabsf(s) > kSteepest ? copysignf(kSteepest, s) : s;
}
__device__ __forceinline__ int bias_from(const Sight &x, int p, int sinks)
{
    const int hi = x.lo < x.hi || x.hi < sinks ? x.hi : sinks;  // of the sinks where the window leaves nothing
    const int q = p > x.lo ? p : x.lo;
    return q < hi - 1 ? q : hi - 1;
}

// An infinity or a NaN among the values of a key that some rows of a workgroup attend to reaches
// its other rows through the matrix product, 0 x infinity being NaN. Where a workgroup's sums came
// out so and such a key holds such a value, its rows are computed again here, one by one and without
// the matrix cores, each from the keys that it attends to and no others. Returns whether it was so.
// (Looking through the values of tiles that rows see in part, before use, cost 2 to 6 % of every
// call; this costs nothing measurable until it is needed, and much then: a NaN among the last
// values of a prompt of 8,192 tokens on 8,192, 1.1 ms to 196 ms, which is one workgroup's 256 rows.)
template <typename T, int D, int MODE>
__device__ __forceinline__ bool repair(const AttnArgs &a, const std::conditional_t<MODE != kPlain, RowRangeEx, RowRange> &in_lds, int *found,
                                       float *part, float2 *part_ml)
{
    const auto x = in_lds;
    constexpr bool EX = MODE != kPlain;
    constexpr int EL = sizeof(T), ROWB = D * EL, PPR = ROWB / 16, PL = D / 64;  // PL: channels of a lane
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, G = static_cast<int>(a.by_group.d);
    const AttnStream s = attn_stream(a, x.b);
    const int end = s.len + (a.k ? s.n : 0), page = 1 << a.page_shift, prefix = EX ? prefix_of(a, x.b, end) : 0;
    auto row_of = [&](int j, const void *pool, const void *own, int64_t stride) -> const T * {  // NULL: no such key
        if (j >= s.len)
            return j < end ? static_cast<const T *>(own) + (s.row0 + j - s.len) * stride + static_cast<int64_t>(x.kvh) * D : nullptr;
        const int id = a.table[static_cast<int64_t>(x.b) * a.max_pages + (j >> a.page_shift)];
        return id >= 0 && id < a.num_pages
                   ? static_cast<const T *>(pool) + ((static_cast<int64_t>(id) * a.KV + x.kvh) * page + (j & (page - 1))) * D
                   : nullptr;
    };
    float sum = 0.f;
    auto look = [&](int from, int to) {  // a piece of a value row per lane and turn
        for (int64_t i = threadIdx.x; i < static_cast<int64_t>(to - from) * PPR; i += 64 * x.nwaves)
            if (const T *v = row_of(from + static_cast<int>(i / PPR), a.vp, a.v, a.v_stride))
                for (int e = 0; e < 16 / EL; ++e)
                    sum = fmaf(static_cast<float>(v[i % PPR * (16 / EL) + e]), 0.f, sum);
    };
    if constexpr (EX) {
        // a key that some rows attend to and not all is below the largest of their lower bounds, or
        // from the least of their upper ones on; no row attends to one from hi_max on
        const Bounds &y = x.bounds;
        auto up_to = [&](int v) { return v < y.hi_max ? v : y.hi_max; };
        look(y.lo_min, up_to(y.lo_max));
        look(y.hi_min, y.hi_max);
        if (a.sinks > 0)
            look(y.f_min, up_to(y.f_max < a.sinks ? y.f_max : a.sinks));
    } else {
        const Sight first = sight_of<EX>(a, s, end, 0, a.by_group(x.r_first)), last = sight_of<EX>(a, s, end, 0, a.by_group(x.r_end - 1));
        look(first.lo, last.lo);
        look(first.hi, last.hi);
    }
    const int mine = __ballot(sum != sum) != 0;
    if (lane == 0)
        found[w] = mine;
    __syncthreads();
    int any = 0;
    for (int i = 0; i < x.nwaves; ++i)
        any |= found[i];
    if (!__builtin_amdgcn_readfirstlane(any))
        return false;
    const float sc = EX ? 1.f : a.scale * kLog2e;
    for (int row = x.r_first + w; row < x.r_end; row += x.nwaves) {
        const int tok = a.by_group(row), head = x.kvh * G + row - tok * G;
        const Sight see = sight_of<EX>(a, s, end, prefix, tok);
        const float slope = EX && a.score.slopes ? slope_of(a.score, head) * kLog2e : 0.f;
        const T *q = static_cast<const T *>(a.q) + (s.row0 + tok) * a.q_stride + static_cast<int64_t>(head) * D;
        float m = -__builtin_inff(), l = 0.f, o[PL] = {};
        for (int t = x.t0; t < x.t1; ++t) {
            const bool cached = t < x.ns + x.nw;
            const int first = t < x.ns ? t * x.tk : cached ? (x.w0 + t - x.ns) * x.tk : s.len + (x.c0 + t - x.ns - x.nw) * x.tk;
            const int stop = cached ? s.len : end;
            for (int kk = 0; kk < x.tk; kk += 64) {
                const int j = first + kk + lane;
                const T *k = nullptr, *v = nullptr;
                if (kk + lane < x.tk && j < stop && j < see.hi && (j >= see.lo || (j < a.sinks && j >= see.first))) {
                    k = row_of(j, a.kp, a.k, a.k_stride);
                    v = row_of(j, a.vp, a.v, a.v_stride);
                }
                float sj = 0.f;
                if (k)
                    for (int c = 0; c < D; ++c)
                        sj = fmaf(static_cast<float>(q[c]), static_cast<float>(k[c]), sj);
                if constexpr (EX) {
                    sj = MODE >= kCapped ? capped(sj, a.score) : sj * (a.scale * kLog2e);
                    if (a.score.slopes)
                        sj = fmaf(-slope, fabsf(static_cast<float>(bias_from(see, s.len + tok, a.sinks) - j)), sj);
                }
                float mx = k ? sj * sc : -__builtin_inff();
                for (int y = 1; y < 64; y *= 2)
                    mx = fmaxf(mx, __shfl_xor(mx, y));
                mx = mx > m ? mx + kAbove : m;  // the reference, as in k_attn
                const float f = m == mx ? 1.f : __builtin_amdgcn_exp2f(m - mx);
                // rounded like the weights of the matrix product, before their sum is taken
                const float wt =
                    k ? static_cast<float>(static_cast<T>(__builtin_amdgcn_exp2f(fmaf(sj, sc, mx == -__builtin_inff() ? 0.f : -mx))))
                      : 0.f;
                float all = wt;
                for (int y = 1; y < 64; y *= 2)
                    all += __shfl_xor(all, y);
                m = mx;
                l = fmaf(l, f, all);
                for (int c = 0; c < PL; ++c)
                    o[c] *= f;
                for (uint64_t left = __ballot(k != nullptr); left; left &= left - 1) {
                    const int y = __builtin_ctzll(left);
                    const T *vy = reinterpret_cast<const T *>(__shfl(reinterpret_cast<uintptr_t>(v), y)) + lane * PL;
                    const float wy = __shfl(wt, y);
                    for (int c = 0; c < PL; ++c)
                        o[c] = fmaf(wy, static_cast<float>(vy[c]), o[c]);
                }
            }
        }
        if (x.nsplit == 1) {
            T *out = static_cast<T *>(a.out) + ((s.row0 + tok) * a.H + head) * D + lane * PL;
            for (int c = 0; c < PL; ++c)
                out[c] = static_cast<T>(o[c] * (l > 0.f ? 1.f / l : l));
        } else {
            const int64_t to = ((static_cast<int64_t>(x.b) * a.KV + x.kvh) * x.nsplit + x.split) * a.block_len * G + row;
            if (lane == 0)
                part_ml[to] = make_float2(m, l);
            for (int c = 0; c < PL; ++c)
                part[to * D + lane * PL + c] = o[c];
        }
    }
    return true;
}

template <typename T, int D, int WM, int WK, int TK>
struct AttnCfg {
    static constexpr int NW = WM * WK, THREADS = 64 * NW, RT = 32 * WM;
    static constexpr int TILE_BYTES = TK * Tile<T, D>::ROWB;
};

template <typename T, int D, int WM, int WK, int TK, int WPE, int MODE>
__global__ __launch_bounds__((AttnCfg<T, D, WM, WK, TK>::THREADS))
__attribute__((amdgpu_waves_per_eu(WPE, WPE))) void k_attn(AttnArgs a, AttnPlan pl, float *part, float2 *part_ml,
                                                                      const int *order)
{
    using C = AttnCfg<T, D, WM, WK, TK>;
    using L = Tile<T, D>;
    using Frag = typename L::Frag;
    constexpr int NW = C::NW, ROWB = L::ROWB, PPR = ROWB / 16;
    constexpr int RPC = 1024 / ROWB;                // rows of a copy
    constexpr int NC = C::TILE_BYTES / 1024 / NW;   // copies of a wavefront per tile, of K and of V
    constexpr int PIDS = (TK + 63) / 64;            // 64-key words of a tile's key mask
    constexpr int KB = TK / 32 / WK;                // 32-key blocks of a wavefront per tile
    constexpr int EL = sizeof(T);
    constexpr bool EX = MODE != kPlain;
    // Whether `raise` and `weigh` find raw scores, to be scaled: a bias is then what the products start
    // from. float32 adds it up in up to 64 products, each with its rounding, so there it comes after.
    constexpr bool RAW = MODE == kPlain || (MODE == kRanged && EL == 2);
    constexpr bool POLY = MODE == kCapped && D == 128;  // weights may be made by the cap's polynomial
    constexpr bool SCHED = MODE != kPlain;  // the order of LDS reads and products is given
    constexpr uint64_t kAll = TK < 64 ? 0xffffffffull : ~0ull;  // a mask of keys with all of them
    static_assert(C::TILE_BYTES % (1024 * NW) == 0 && TK % (32 * WK) == 0, "tile shape");

    // one array per stage and operand, so that reads of one need not wait for copies into another
    __shared__ __attribute__((aligned(16))) char k0[C::TILE_BYTES], v0[C::TILE_BYTES], k1[C::TILE_BYTES], v1[C::TILE_BYTES];
    __shared__ float2 ml[WK > 1 ? NW * 32 : 1];
    __shared__ int odd[2][NW];  // what a wavefront found, and this workgroup's part: see repair
    __shared__ std::conditional_t<EX, RowRangeEx, RowRange> mine;
    __shared__ Bounds by_wave[EX ? NW : 1];
    auto KBUF = [&](auto S) -> char * { return S.value == 0 ? k0 : k1; };
    auto VBUF = [&](auto S) -> char * { return S.value == 0 ? v0 : v1; };

    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / WK, wk = w % WK, hf = lane >> 5, l32 = lane & 31;

    // ---- this workgroup's part, row tile and unit (see AttnPlan)
    const int nsplit = pl.nsplit, wid = blockIdx.x >> 3, outer = pl.by_inner(wid), inner = wid - outer * static_cast<int>(pl.by_inner.d);
    const int part_no = (pl.rt_fast ? outer : inner) * 8 + (blockIdx.x & 7);
    if (part_no >= pl.units)
        return;
    const int which = pl.by_units(part_no), u = pl.by_units.rest(part_no);
    const int rt_up = (pl.rt_fast ? inner : outer) * pl.sub + which;
    if (rt_up >= pl.nrt)
        return;
    const int uk = pl.by_kv(u), kvh = pl.by_kv.rest(u), b = pl.by_split(uk), split = pl.by_split.rest(uk);
    int rt = a.block ? pl.nrt - 1 - rt_up : rt_up;  // ordered: the longest ranges first
    if (EX && order)
        rt = __builtin_amdgcn_readfirstlane(order[static_cast<int64_t>(b) * pl.nrt + rt_up]);
    const int G = static_cast<int>(a.by_group.d);
    const int *table = a.table + static_cast<int64_t>(b) * a.max_pages;
    auto page_no = [&](int i) { return a.max_pages > 0 ? table[i < a.max_pages ? i : a.max_pages - 1] : -1; };
    const int first_pages[2] = {page_no(lane), page_no(64 + lane)};
    const AttnStream s = attn_stream(a, b);
    const int rows = s.n * G, r_first = rt * C::RT;
    if (r_first >= rows)
        return;
    const int r_end = r_first + C::RT < rows ? r_first + C::RT : rows;

    // ---- what the workgroup's rows and this wavefront's rows attend to
    const int n = a.k ? s.n : 0, end = s.len + n;  // keys at positions [0, end)
    const int prefix = EX ? prefix_of(a, b, end) : 0;
    auto sight = [&](int tok) { return sight_of<EX>(a, s, end, prefix, tok); };
    const int wr0 = r_first + wm * 32;
    const bool active = wr0 < r_end;
    const int wr1 = wr0 + 31 < r_end ? wr0 + 31 : r_end - 1;
    Bounds wg, wave;  // of the workgroup's rows, of this wavefront's
    if (EX && (a.score.first || a.score.last)) {
        const Sight x = sight(a.by_group(wr0 + l32 < r_end ? wr0 + l32 : r_end - 1));
        wave = Bounds{x.lo, x.lo, x.hi, x.hi, x.first, x.first};
        auto both = [](Bounds v, const Bounds &o) {
            return Bounds{min(v.lo_min, o.lo_min), max(v.lo_max, o.lo_max), min(v.hi_min, o.hi_min),
                          max(v.hi_max, o.hi_max), min(v.f_min, o.f_min), max(v.f_max, o.f_max)};
        };
        auto uniform = [](Bounds v) {
            auto u = [](int y) { return __builtin_amdgcn_readfirstlane(y); };
            return Bounds{u(v.lo_min), u(v.lo_max), u(v.hi_min), u(v.hi_max), u(v.f_min), u(v.f_max)};
        };
#pragma unroll
        for (int y = 1; y < 32; y *= 2)
            wave = both(wave, Bounds{__shfl_xor(wave.lo_min, y), __shfl_xor(wave.lo_max, y), __shfl_xor(wave.hi_min, y),
                                     __shfl_xor(wave.hi_max, y), __shfl_xor(wave.f_min, y), __shfl_xor(wave.f_max, y)});
        wave = uniform(wave);
        if (lane == 0)
            by_wave[w] = wave;
        __syncthreads();
        wg = by_wave[0];
#pragma unroll
        for (int i = 1; i < NW; ++i)
            wg = both(wg, by_wave[i]);
        wg = uniform(wg);
    } else {  // bounds grow with the token
        const Sight x = sight(a.by_group(r_first)), y = sight(a.by_group(r_end - 1));
        wg = Bounds{x.lo, y.lo, x.hi, y.hi, x.first, y.first};
        const Sight wx = sight(a.by_group(wr0)), wy = sight(a.by_group(wr1));
        wave = Bounds{wx.lo, wy.lo, wx.hi, wy.hi, wx.first, wy.first};
    }
    const int lo_min = wg.lo_min, lo_max = wg.lo_max, hi_min = wg.hi_min, hi_max = wg.hi_max;

    // ---- tiles: sinks outside the window, the cached window, the chunk's own keys
    const int len = !EX || s.len < hi_max ? s.len : hi_max;  // cached tokens to be walked
    const int sink_len = a.window ? (a.sinks < len ? a.sinks : len) : 0;
    const int len_tiles = (len + TK - 1) / TK, w0 = lo_min < len ? lo_min / TK : len_tiles, nw = len_tiles - w0;
    const int sink_tiles = (sink_len + TK - 1) / TK, ns = sink_tiles < w0 ? sink_tiles : w0;
    const int c_lo = a.sinks > s.len || lo_min <= s.len ? 0 : lo_min - s.len, c_hi = hi_max - s.len;  // c_hi may be <= c_lo
    const int c0 = c_lo / TK, nc = n > 0 && c_hi > c_lo ? (c_hi + TK - 1) / TK - c0 : 0;
    const int nt = ns + nw + nc;
    const int per = pl.by_split(nt + nsplit - 1), t0 = split * per, t1 = t0 + per < nt ? t0 + per : nt;

    const bool differ = lo_min != lo_max || hi_min != hi_max || (EX && wg.f_min != wg.f_max);  // some rows see what others do not
    if (differ && threadIdx.x == 0) {
        static_cast<RowRange &>(mine) = RowRange{b, kvh, split, nsplit, r_first, r_end, t0, t1, ns, nw, w0, c0, TK, NW};
        if constexpr (EX)
            mine.bounds = wg;
    }

    struct Cursor {
        int t, start;  // tile, and its first key: cached position or index into the chunk
        bool cached;
    };
    auto at = [&](int t) {
        return t < ns        ? Cursor{t, t * TK, true}
               : t < ns + nw ? Cursor{t, (w0 + t - ns) * TK, true}
                             : Cursor{t, (c0 + t - ns - nw) * TK, false};
    };
    auto advance = [&](Cursor &x) {
        ++x.t;
        x.start += TK;
        if (x.t == ns || x.t == ns + nw)
            x = at(x.t);
    };

    // ---- copies
    const int page = 1 << a.page_shift, last_page = (s.len > 0 ? s.len - 1 : 0) >> a.page_shift;
    const int page_bytes = page * ROWB;
    const uint32_t pool_step = static_cast<uint32_t>(a.KV * page_bytes);  // from page to page
    // Pages: lane i holds the offset in its pool of page pbase + i (pbase a multiple of 64, so
    // that no tile straddles it), and in `next` the number of the one 64 pages on. The first 64
    // are loaded along with the stream's length, before it is known whether they are needed.
    int pbase = -1, next = first_pages[1];
    uint32_t page_lo = 0, page_hi = 0;
    uint64_t held = 0, whole_pages = 0;  // which of the 64 are pages of the pool; or past the stream's last
    auto find_pages = [&](int start) {
        const int p = (start >> a.page_shift) & ~63;
        if (p != pbase) {
            const uint32_t id = p == 0 ? first_pages[0] : p == pbase + 64 ? next : page_no(p + lane);
            if (p != 0)
                next = page_no(p + 64 + lane);
            pbase = p;
            held = __ballot(id < static_cast<uint32_t>(a.num_pages));
            whole_pages = held | __ballot(p + lane > last_page);
            const uint64_t off = static_cast<uint64_t>(id) * pool_step;
            page_lo = static_cast<uint32_t>(off), page_hi = static_cast<uint32_t>(off >> 32);
        }
    };
    const int crow = lane / PPR, cslot = lane % PPR;  // row of a copy, LDS piece of that row
    const char *kp = static_cast<const char *>(a.kp) + static_cast<int64_t>(kvh) * page_bytes;
    const char *vp = static_cast<const char *>(a.vp) + static_cast<int64_t>(kvh) * page_bytes;
    const char *ck = static_cast<const char *>(a.k) + (s.row0 * a.k_stride + static_cast<int64_t>(kvh) * D) * EL;
    const char *cv = static_cast<const char *>(a.v) + (s.row0 * a.v_stride + static_cast<int64_t>(kvh) * D) * EL;
    uint64_t valid[2][PIDS];  // per stage: the tile's keys that exist and that some row attends to,
    int jpos[2];              // and the position of its first key
    auto copy = [&](auto S, const Cursor &x) {
        jpos[S.value] = x.cached ? x.start : s.len + x.start;
        if (x.cached)
            find_pages(x.start);
        if (x.cached && x.start + TK <= s.len && x.start >= lo_min && (!EX || x.start + TK <= hi_max) && whole_pages == ~0ull) {
#pragma unroll
            for (int i = 0; i < PIDS; ++i)
                valid[S.value][i] = kAll;
        } else {
#pragma unroll
            for (int i = 0; i < PIDS; ++i) {
                const int kk = 64 * i + lane, j = jpos[S.value] + kk;
                const bool there = x.cached ? (j < s.len) & ((held >> ((j >> a.page_shift) & 63)) & 1) : j < end;
                const bool visible = (j < hi_max) & ((j >= lo_min) | (j < a.sinks)) & (!EX || j >= wg.f_min);
                valid[S.value][i] = __ballot((kk < TK) & there & visible);
            }
        }
        if (x.cached) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int row0 = (w + NW * c) * RPC, row = row0 + crow;
                const int pi = ((x.start + row0) >> a.page_shift) & 63, slot = (x.start + row0) & (page - 1);
                const bool ok = (held >> pi) & 1;  // not held: an empty range, nothing is read
                const uint64_t base = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(page_hi, pi))) << 32 |
                                      static_cast<uint32_t>(__builtin_amdgcn_readlane(page_lo, pi));
                const int off = slot * ROWB + crow * ROWB;
                copy_to_lds(buffer_range(kp + base, ok ? page_bytes : 0), KBUF(S) + row0 * ROWB,
                            off + (cslot ^ L::swz_k(row)) * 16);
                copy_to_lds(buffer_range(vp + base, ok ? page_bytes : 0), VBUF(S) + row0 * ROWB,
                            off + (cslot ^ L::swz_v(row)) * 16);
            }
        } else {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int row0 = (w + NW * c) * RPC, row = row0 + crow;
                // rows past the chunk's end: its last row again
                const int i0 = x.start + row0 < n ? x.start + row0 : n - 1;
                const int dr = i0 + crow < n ? crow : n - 1 - i0;
                copy_to_lds(buffer_range(ck + i0 * a.k_stride * EL, 0x7fffffff), KBUF(S) + row0 * ROWB,
                            dr * static_cast<int>(a.k_stride) * EL + (cslot ^ L::swz_k(row)) * 16);
                copy_to_lds(buffer_range(cv + i0 * a.v_stride * EL, 0x7fffffff), VBUF(S) + row0 * ROWB,
                            dr * static_cast<int>(a.v_stride) * EL + (cslot ^ L::swz_v(row)) * 16);
            }
        }
    };
    Cursor nx = at(t0);  // the tile to be copied next
    auto start = [&](auto S) {
        copy(S, nx);
        advance(nx);
    };

    // ---- queries: B operands, one row per lane
    Frag q[L::STEPS];
    const int my_row = wr0 + l32 < r_end ? wr0 + l32 : r_end - 1, tok = a.by_group(my_row), head = kvh * G + my_row - tok * G;
    const Sight my = sight(tok);
    const int p_hi = my.hi, p_lo = my.lo;  // attends to [p_lo, p_hi) and below a.sinks
    const T *q_row = static_cast<const T *>(a.q) + (s.row0 + tok) * a.q_stride + static_cast<int64_t>(head) * D;
#pragma unroll
    for (int st = 0; st < L::STEPS; ++st)
        q[st] = *reinterpret_cast<const Frag *>(q_row + (2 * st + hf) * (16 / EL));

    f32x16 o[D / 32] = {};
    float m = -__builtin_inff(), l = 0.f;
    const float sc = RAW ? a.scale * kLog2e : 1.f;  // of scores as `raise` and `weigh` find them
    const bool bias = EX && a.score.slopes;
    float slope = bias ? slope_of(a.score, head) * (RAW ? 1.f / a.scale : kLog2e) : 0.f;
    const int from = bias_from(my, s.len + tok, a.sinks) - 4 * hf;

    // ---- operand reads. Every lane offset is one opaque value, a single step from its array:
    // the compiler then sees which array a read is from, and does not make it wait for copies
    // into the others.
    int koff[L::STEPS], voff[sizeof(T) == 2 ? D / 32 : 1];
#pragma unroll
    for (int st = 0; st < L::STEPS; ++st) {
        koff[st] = (32 * wk * KB + l32) * ROWB + (((2 * st + hf) ^ L::swz_k(l32)) * 16);
        asm volatile("" : "+v"(koff[st]));
    }
    if constexpr (EL == 2) {
        const int j16 = lane & 15, cg = (lane >> 4) & 1;  // lane of a 16-lane group, column half
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
            const int pc = (4 * d + 2 * cg + ((j16 & 3) >> 1)) ^ L::swz_v(j16 >> 2);
            voff[d] = (32 * wk * KB + 4 * hf + (j16 >> 2)) * ROWB + pc * 16 + (j16 & 1) * 8;
            asm volatile("" : "+v"(voff[d]));
        }
    } else {
        voff[0] = (32 * wk * KB + 4 * hf) * ROWB + l32 * 4;
        asm volatile("" : "+v"(voff[0]));
    }

    // ---- one tile: this wavefront's KB blocks of 32 keys
    f32x16 sv[KB];               // scores
    // the bias of block kb's key r of a lane: -slope |from - j|. Keys of the cache that a row sees are
    // not past `from` (either `from` is the row's own position or later, or it is its last key)
    const bool steep = MODE == kRanged && RAW && bias && __ballot(fabsf(slope) * a.scale * static_cast<float>(end) > kSteepest) != 0;
    auto biased = [&](auto S, int kb, auto with) {
        const int d = from - jpos[S.value] - 32 * (wk * KB + kb);
        if (steep) {
            float scale = a.scale;
            asm volatile("" : "+v"(scale));  // made here, not kept through the loop
            const float least = -kSteepest / scale;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                sv[kb][r] = with(fmaxf(-slope * fabsf(static_cast<float>(d - 8 * (r / 4) - r % 4)), least), r);
        } else if (jpos[S.value] < s.len) {
            // key r is 8 (r / 4) + r % 4 further on. In steps of 1, 2 and 4 slopes, which instructions
            // hold themselves; other factors would take a register each
            float b = -slope * static_cast<float>(d);
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const float b1 = b + slope;
                sv[kb][r] = with(b, r);
                sv[kb][r + 1] = with(b1, r + 1);
                sv[kb][r + 2] = with(fmaf(slope, 2.f, b), r + 2);
                sv[kb][r + 3] = with(fmaf(slope, 2.f, b1), r + 3);
                b = fmaf(slope, 4.f, fmaf(slope, 4.f, b));
            }
        } else {
            float far = static_cast<float>(d);
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const float far1 = far - 1.f;
                sv[kb][r] = with(-slope * fabsf(far), r);
                sv[kb][r + 1] = with(-slope * fabsf(far1), r + 1);
                sv[kb][r + 2] = with(-slope * fabsf(far - 2.f), r + 2);
                sv[kb][r + 3] = with(-slope * fabsf(far1 - 2.f), r + 3);
                far = far - 4.f - 4.f;
            }
        }
    };
    auto scores = [&](auto S) {  // S^T = K Q^T
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            sv[kb] = f32x16{};
            if (MODE == kRanged && RAW && bias)
                biased(S, kb, [](float b, int) { return b; });
        }
        auto read = [&](int i) {
            return *reinterpret_cast<const Frag *>(&KBUF(S)[koff[i % L::STEPS] + 32 * (i / L::STEPS) * ROWB]);
        };
        constexpr int N = KB * L::STEPS;
        if constexpr (SCHED) {
            // GS operands are read while the GS in front of them are multiplied. Left to itself the
            // compiler kept one, and waited for LDS in front of every product
            constexpr int GS = EL == 2 && D == 128 ? 4 : 2;
            Frag kf[2][GS];
#pragma unroll
            for (int i = 0; i < GS; ++i)
                kf[0][i] = read(i);
#pragma unroll
            for (int g = 0; g < N / GS; ++g) {
#pragma unroll
                for (int i = 0; i < GS && g + 1 < N / GS; ++i)
                    kf[(g + 1) & 1][i] = read((g + 1) * GS + i);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < GS; ++i) {
                    const int at = g * GS + i;
                    sv[at / L::STEPS] = L::qk(kf[g & 1][i], q[at % L::STEPS], sv[at / L::STEPS]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                sv[i / L::STEPS] = L::qk(read(i), q[i % L::STEPS], sv[i / L::STEPS]);
        }
    };
    auto hide = [&](auto S) {  // scores of what the query does not attend to: -infinity
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int blk = wk * KB + kb, jb = jpos[S.value] + 32 * blk;
            const uint32_t bits = static_cast<uint32_t>((blk < 2 ? valid[S.value][0] : valid[S.value][PIDS - 1]) >> (32 * (blk & 1)));
            // the block's keys that the query attends to, from the lane's first on
            uint32_t see = bits & below(p_hi - jb) & (~below(p_lo - jb) | below(a.sinks - jb));
            if constexpr (EX)
                see &= ~below(my.first - jb);
            see >>= 4 * hf;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const uint32_t on = __builtin_amdgcn_sbfe(see, 8 * (r / 4) + r % 4, 1);  // all bits or none
                sv[kb][r] = __uint_as_float((__float_as_uint(sv[kb][r]) & on) | (0xff800000u & ~on));
            }
        }
    };
    const Poly poly = {a.score.q[0], a.score.q[1], a.score.q[2], a.score.q[3]};
    auto largest = [&]() {  // magnitude of a lane's scores; a NaN does not count
        float top = 0.f;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                top = fmaxf(top, fabsf(sv[kb][r]));
        return top;
    };
    // scores as `weigh` takes them, where the products do not leave them so
    auto shape = [&](auto S) {
        if constexpr (MODE >= kCapped) {
            auto each = [&](auto f) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        sv[kb][r] = f(sv[kb][r]);
            };
            if constexpr (MODE == kCapped)
                each([&](float x) { return capped_any(x, a.score); });
            else if (EL == 4 && __ballot(largest() * a.score.x_per_score > 0.6f) == 0)
                each([&](float x) { return capped_near(x, a.score); });
            else
                each([&](float x) { return capped(x, a.score); });
        } else {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                sv[kb] *= a.scale * kLog2e;
        }
        if (bias) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                biased(S, kb, [&](float b, int r) { return sv[kb][r] + b; });
        }
    };
    // Form 1: the weights take raw scores through the tile's polynomial; 0: scores times sc.
    // The query's new reference (a lane holds half of its keys; the other half's lane has the rest)
    auto raise = [&](auto form) {
        float mx = sv[0][0];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                mx = fmaxf(mx, sv[kb][r]);
        mx = half_max(mx);
        if constexpr (form.value == 1)
            mx *= poly(mx);
        else
            mx *= sc;
        if (__ballot(mx > m)) {
            const float mn = fmaxf(m, mx + kAbove);
            const float f = m == mn ? 1.f : __builtin_amdgcn_exp2f(m - mn);  // equal infinities: 1
            m = mn;
            l *= f;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
                o[d] *= f;
        }
    };
    // weights, and O^T += V^T P^T one part of 16 keys behind them, so that a wavefront's products
    // and exponentials overlap
    auto weigh = [&](auto S, auto form) {
        constexpr int PARTS = 2 * KB;
        const float ref = m == -__builtin_inff() ? 0.f : m;
        auto power = [&](float x) { return form.value == 1 ? fmaf(x, poly(x), -ref) : fmaf(x, sc, -ref); };
        float wt[PARTS][8];
        bf16x8 wb[PARTS];
        auto make = [&](int x, int from, int to) {
#pragma unroll
            for (int e = from; e < to; ++e)
                wt[x][e] = __builtin_amdgcn_exp2f(power(sv[x / 2][8 * (x % 2) + e]));
        };
        auto add = [&](int x) {
            if constexpr (EL == 2) {
                // the sum is of the rounded weights, two per instruction
                wb[x] = to_bf16x8(wt[x]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    l = add_pair(wb[x], e, l);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    l += wt[x][e];
            }
        };
        auto read = [&](int x, int d) {  // values of part x, channels of block d
            const int at = voff[d] + 16 * x * ROWB;
            return cat(tr_read(reinterpret_cast<const __bf16 *>(&VBUF(S)[at])),
                       tr_read(reinterpret_cast<const __bf16 *>(&VBUF(S)[at + 8 * ROWB])));
        };
        if constexpr (SCHED && EL == 4) {
            // values of four keys are read while the four in front of them are multiplied, the next
            // part's weights made between the products
            constexpr int DB = D / 32;
            float vf[2][4][DB];
            auto read_four = [&](int g) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        vf[g & 1][e][d] = *reinterpret_cast<const float *>(&VBUF(S)[voff[0] + (8 * g + e) * ROWB + 128 * d]);
            };
            read_four(0);
            make(0, 0, 8);
            add(0);
#pragma unroll
            for (int g = 0; g < 2 * PARTS; ++g) {
                if (g + 1 < 2 * PARTS)
                    read_four(g + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(vf[g & 1][e][d], wt[g / 2][4 * (g & 1) + e], o[d], 0, 0, 0);
                    if (g / 2 + 1 < PARTS)
                        make(g / 2 + 1, 4 * (g & 1) + e, 4 * (g & 1) + e + 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (g % 2 == 1 && g / 2 + 1 < PARTS)
                    add(g / 2 + 1);
            }
        } else if constexpr (SCHED) {
            // A part's values are read while weights are made. At headdim 128 two wavefronts share a
            // SIMD: there they are read a part ahead, and a product is followed by a share of the next
            // part's weights; at 64 the four of a SIMD cover each other, and registers are short.
            constexpr int DB = D / 32;
            constexpr bool AHEAD = D == 128;
            bf16x8 vf[AHEAD ? 2 : 1][DB];
            auto read_all = [&](int x) {
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    vf[AHEAD ? x & 1 : 0][d] = read(x, d);
                __builtin_amdgcn_sched_barrier(0);
            };
            auto multiply = [&](int x, int d) {
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[AHEAD ? x & 1 : 0][d], wb[x], o[d], 0, 0, 0);
            };
#pragma unroll
            for (int x = 0; x < PARTS; ++x) {
                if (AHEAD || x > 0)
                    read_all(AHEAD ? x : x - 1);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    if (AHEAD && x > 0)
                        multiply(x - 1, d);
                    make(x, 8 * d / DB, 8 * (d + 1) / DB);
                    if (AHEAD)
                        __builtin_amdgcn_sched_barrier(0);
                }
                add(x);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int d = 0; d < DB && !AHEAD && x > 0; ++d)
                    multiply(x - 1, d);
            }
            if (!AHEAD)
                read_all(PARTS - 1);
#pragma unroll
            for (int d = 0; d < DB; ++d)
                multiply(PARTS - 1, d);
        } else {
#pragma unroll
            for (int x = 0; x <= PARTS; ++x) {
                if (x < PARTS) {
                    make(x, 0, 8);
                    add(x);
                }
                if (x > 0) {
                    if constexpr (EL == 2) {
#pragma unroll
                        for (int d = 0; d < D / 32; ++d)
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read(x - 1, d), wb[x - 1], o[d], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
#pragma unroll
                            for (int d = 0; d < D / 32; ++d) {
                                const int at = voff[0] + (16 * (x - 1) + 8 * (e / 4) + e % 4) * ROWB + 128 * d;
                                o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(*reinterpret_cast<const float *>(&VBUF(S)[at]),
                                                                            wt[x - 1][e], o[d], 0, 0, 0);
                            }
                    }
                }
            }
        }
    };

    // whether this wavefront has anything to do in the tile of stage S, and whether its rows see it whole
    auto seen = [&](auto S) {
        const int j0 = jpos[S.value];
        return active && j0 < wave.hi_max && (j0 + TK > wave.lo_min || j0 < a.sinks);
    };
    auto full = [&](auto S) {
        bool all = true;
#pragma unroll
        for (int i = 0; i < PIDS; ++i)
            all = all && valid[S.value][i] == kAll;
        return all;
    };
    auto whole = [&](auto S) {
        const int j0 = jpos[S.value];
        return full(S) && j0 + TK <= wave.hi_min && (j0 >= wave.lo_max || (j0 + TK <= a.sinks && (!EX || j0 >= wave.f_max)));
    };
    auto clear_absent = [&](auto S) {  // this thread's share of the values no row attends to
#pragma unroll
        for (int x = 0; x < C::TILE_BYTES / 16 / C::THREADS; ++x) {
            const int piece = x * C::THREADS + threadIdx.x, row = piece / PPR;
            if (!((valid[S.value][PIDS == 1 ? 0 : row >> 6] >> (row & 63)) & 1))
                *reinterpret_cast<uint4 *>(&VBUF(S)[piece * 16]) = make_uint4(0, 0, 0, 0);
        }
    };

    // the queries' loads end here, not at their first use inside the loop, where the wait for them
    // would be one for the copies in flight too
#pragma unroll
    for (int st = 0; st < L::STEPS; ++st)
        asm volatile("" : "+v"(q[st]));
    if constexpr (EX)
        asm volatile("" : "+v"(slope));

    // ---- the loop over tiles: iteration t waits for tile t (its own copies, then everyone's),
    // starts the copies of the next tile into the stage that was last read before the barrier,
    // and computes
    auto step = [&](auto S, int t) {
        workgroup_lds_barrier<0>();
        if (!full(S)) {  // the same for every wavefront
            clear_absent(S);
            workgroup_lds_barrier<63>();
        }
        if (t + 1 < t1)
            start(Int<1 - S.value>{});
        if (seen(S)) {
            scores(S);
            if constexpr (POLY) {
                const bool all = whole(S), small = !bias && all && __ballot(largest() > a.score.half_cap) == 0;
                if (small) {
                    raise(Int<1>{});
                    weigh(S, Int<1>{});
                    return;
                }
                shape(S);
                if (!all)
                    hide(S);
            } else {
                if constexpr (!RAW)
                    shape(S);
                if (!whole(S))
                    hide(S);
            }
            raise(Int<0>{});
            weigh(S, Int<0>{});
        }
    };
    if (t0 < t1)
        start(Int<0>{});
    for (int t = t0; t < t1; t += 2) {
        step(Int<0>{}, t);
        if (t + 1 < t1)
            step(Int<1>{}, t + 1);
    }
    l = half_sum(l);

    // ---- repair: an infinity or a NaN among the values of a key that some of the workgroup's rows
    // attend to has reached its other rows too, 0 x infinity being NaN
    if (differ) {
        float sum = 0.f;  // 0 x an infinity or a NaN is NaN
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                sum = fmaf(o[d][r], 0.f, sum);
        if (anyone<NW>(odd[0], sum != sum)) {
            // what it needs comes from the kernel's argument memory and from LDS again, so that
            // nothing is kept in registers for it through the loop
            auto *args = (const AttnArgs *)__builtin_amdgcn_kernarg_segment_ptr();
            asm volatile("" : "+s"(args));
            if (repair<T, D, MODE>(*args, mine, odd[1], part, part_ml))
                return;
        }
    }

    // ---- wavefronts that shared the rows: join in LDS, in wavefront order
    if constexpr (WK > 1) {
        constexpr int UNIT = 32 * D * 4, PER = C::TILE_BYTES / UNIT;  // bytes of 32 rows; units per array
        static_assert((WK - 1) * WM <= 4 * PER, "the stages hold the partial rows");
        auto unit = [&](int x) {  // the x-th other wavefront's rows
            const int i = (x - 1) * WM + wm;
            char *arr = i / PER == 0 ? k0 : i / PER == 1 ? v0 : i / PER == 2 ? k1 : v1;
            return reinterpret_cast<f32x4 *>(arr + (i % PER) * UNIT);
        };
        __syncthreads();
        if (hf == 0)
            ml[w * 32 + l32] = make_float2(m, l);
        if (wk > 0) {
            f32x4 *to = unit(wk);
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    to[(d * 4 + r) * 64 + lane] = f32x4{o[d][4 * r], o[d][4 * r + 1], o[d][4 * r + 2], o[d][4 * r + 3]};
        }
        __syncthreads();
        if (wk > 0)
            return;
        const float own = m;
#pragma unroll
        for (int x = 1; x < WK; ++x)
            m = fmaxf(m, ml[(w + x) * 32 + l32].x);
        const float f0 = own == m ? 1.f : __builtin_amdgcn_exp2f(own - m);
        l *= f0;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
            o[d] *= f0;
#pragma unroll
        for (int x = 1; x < WK; ++x) {
            const float2 v = ml[(w + x) * 32 + l32];
            const float f = v.x == m ? 1.f : __builtin_amdgcn_exp2f(v.x - m);
            l = fmaf(v.y, f, l);
            const f32x4 *from = unit(x);
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const f32x4 ov = from[(d * 4 + r) * 64 + lane];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[d][4 * r + e] = fmaf(ov[e], f, o[d][4 * r + e]);
                }
        }
    }

    // ---- rows out: normalized, or partial with their maximum and sum
    if (wr0 + l32 >= r_end)
        return;
    if (nsplit == 1) {
        const float inv = l > 0.f ? 1.f / l : l;  // nothing attended to: 0; NaN stays
        T *out = static_cast<T *>(a.out) + ((s.row0 + tok) * a.H + head) * D + 4 * hf;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const f32x4 ov = f32x4{o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]} * inv;
                if constexpr (EL == 2)
                    *reinterpret_cast<bf16x4 *>(out + 32 * d + 8 * x) = __builtin_convertvector(ov, bf16x4);
                else
                    *reinterpret_cast<f32x4 *>(out + 32 * d + 8 * x) = ov;
            }
    } else {
        const int64_t R = static_cast<int64_t>(a.block_len) * G;
        const int64_t at = ((static_cast<int64_t>(b) * a.KV + kvh) * nsplit + split) * R + wr0 + l32;
        if (hf == 0)
            part_ml[at] = make_float2(m, l);
        float *out = part + at * D + 4 * hf;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<f32x4 *>(out + 32 * d + 8 * x) =
                    f32x4{o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]};
    }
}

// Joins the partial rows of a split cache: out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
// D/4 lanes hold a row, and GROUPS such groups of a workgroup take every GROUPS-th range, joined
// in LDS in group order: many ranges of few rows are read by as many lanes as few of many.
// A range that attended to nothing (sum 0) counts with weight 0: its rows were written.
template <typename T, int D, int GROUPS>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, int nsplit, const float *part, const float2 *part_ml)
{
    constexpr int LPR = D / 4, RPW = 256 / LPR / GROUPS;  // lanes of a row, rows of a workgroup
    __shared__ f32x4 so[GROUPS > 1 ? 256 : 1];
    __shared__ float2 sml[GROUPS > 1 ? 256 : 1];
    const int b = blockIdx.z, kvh = blockIdx.y, G = static_cast<int>(a.by_group.d);
    const int lr = threadIdx.x % LPR, g = threadIdx.x / LPR % GROUPS;
    const int r = blockIdx.x * RPW + threadIdx.x / LPR / GROUPS, c = 4 * lr;
    const AttnStream s = attn_stream(a, b);
    const bool mine = r < s.n * G;
    const int64_t R = static_cast<int64_t>(a.block_len) * G, u0 = (static_cast<int64_t>(b) * a.KV + kvh) * nsplit * R + r;
    float M = -__builtin_inff(), l = 0.f;
    f32x4 o = {};
    if (mine) {
#pragma unroll 4
        for (int x = g; x < nsplit; x += GROUPS)
            M = fmaxf(M, part_ml[u0 + x * R].x);
#pragma unroll 4
        for (int x = g; x < nsplit; x += GROUPS) {
            const float2 v = part_ml[u0 + x * R];
            const f32x4 ov = *reinterpret_cast<const f32x4 *>(part + (u0 + x * R) * D + c);
            const float f = v.x == M ? 1.f : __builtin_amdgcn_exp2f(v.x - M);
            l = fmaf(v.y, f, l);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = fmaf(ov[e], f, o[e]);
        }
    }
    if constexpr (GROUPS > 1) {
        so[threadIdx.x] = o;
        sml[threadIdx.x] = make_float2(M, l);
        __syncthreads();
        if (g > 0)
            return;
        const int first = threadIdx.x;
#pragma unroll
        for (int x = 1; x < GROUPS; ++x)
            M = fmaxf(M, sml[first + x * LPR].x);
        const float f0 = sml[first].x == M ? 1.f : __builtin_amdgcn_exp2f(sml[first].x - M);
        l *= f0;
        o *= f0;
#pragma unroll
        for (int x = 1; x < GROUPS; ++x) {
            const float2 v = sml[first + x * LPR];
            const f32x4 ov = so[first + x * LPR];
            const float f = v.x == M ? 1.f : __builtin_amdgcn_exp2f(v.x - M);
            l = fmaf(v.y, f, l);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = fmaf(ov[e], f, o[e]);
        }
    }
    if (!mine)
        return;
    const float inv = l > 0.f ? 1.f / l : l;
    o *= inv;
    const int tok = a.by_group(r);
    T *out = static_cast<T *>(a.out) + ((s.row0 + tok) * a.H + kvh * G + r - tok * G) * D + c;
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<bf16x4 *>(out) = __builtin_convertvector(o, bf16x4);
    else
        *reinterpret_cast<f32x4 *>(out) = o;
}

template <typename T, int D, int GROUPS>
void join(const AttnArgs &a, int nsplit, const float *part, const float2 *ml, hipStream_t st)
{
    constexpr int RPW = 256 / (D / 4) / GROUPS;
    const int64_t R = static_cast<int64_t>(a.block_len) * (a.H / a.KV);
    k_attn_join<T, D, GROUPS><<<dim3(static_cast<unsigned>((R + RPW - 1) / RPW), a.KV, a.batch), 256, 0, st>>>(a, nsplit, part, ml);
}

// f(WM, WK, TK, WPE): the kernel shape for R rows per (stream, KV head): row blocks of 32 and key
// parts of a workgroup, keys of a tile, wavefronts per SIMD.
//  bf16   up to 64 rows: 2 x 2 (16 rows a head group, 8 streams of 32,768, headdim 128: 107 us,
//         115 us as 8 x 1); more: 8 x 1 (128 rows, headdim 64: 62 us, 77 us as 2 x 2). Up to 32 rows
//         as 1 x 4 with tiles of 128 is no faster: 6 rows on 255 keys 8.4 us, 8.9 so, on 1,000 keys
//         of headdim 128 12.1, 15.6 so, on 16,384 keys the same. More, where rows have ranges of
//         their own: 4 x 1, which waste less at a document's borders (8,191 tokens of 16 heads over 4
//         in documents of 700: 41 us, 47 as 8 x 1; headdim 128 60 and 67; in one document 194 and
//         207, at headdim 128 307 and 297)
//  f32    up to 32 rows of headdim 64: 1 x 4 (32 rows, 8 streams of 4,096: 28 us, 32 us as 2 x 2,
//         47 us as 4 x 1); up to 64 rows: 2 x 2 (64 rows: 34 us, 49 us as 4 x 1; headdim 128:
//         58 us, 83 us); more: 4 x 1, whose products leave no room for more wavefronts
template <typename T, int D, typename F>
auto by_rows(int64_t R, bool ranged, F f)
{
    if constexpr (sizeof(T) == 2) {
        if (R <= 64)
            return f.template operator()<T, D, 2, 2, 64, (D == 64 ? 3 : 2)>();
        if (ranged)
            return f.template operator()<T, D, 4, 1, 64, (D == 64 ? 3 : 2)>();
        return f.template operator()<T, D, 8, 1, 64, (D == 64 ? 4 : 2)>();
    } else {
        if constexpr (D == 64) {
            if (R <= 32)
                return f.template operator()<T, D, 1, 4, 128, 1>();
        }
        if (R <= 64)
            return f.template operator()<T, D, 2, 2, 64, (D == 64 ? 2 : 1)>();
        return f.template operator()<T, D, 4, 1, (D == 64 ? 64 : 32), 2>();
    }
}

template <int MODE>
struct Launch {
    const AttnArgs &a;
    const AttnPlan &p;
    void *ws;
    hipStream_t st;
    template <typename T, int D, int WM, int WK, int TK, int WPE>
    hipError_t operator()() const
    {
        // not built: float32 is exact, and plain rows have no ranges
        constexpr bool never = (MODE == kCapped && sizeof(T) == 4) || (MODE == kPlain && sizeof(T) == 2 && WM == 4);
        if constexpr (never)
            return hipErrorInvalidValue;
        else
            return launch<T, D, WM, WK, TK, WPE>();
    }
    template <typename T, int D, int WM, int WK, int TK, int WPE>
    hipError_t launch() const
    {
        using C = AttnCfg<T, D, WM, WK, TK>;
        float2 *ml = static_cast<float2 *>(ws);
        float *part = reinterpret_cast<float *>(static_cast<char *>(ws) + p.ml_bytes);
        int *order = nullptr;
        if constexpr (MODE != kPlain) {
            if (p.order_bytes > 0) {
                order = reinterpret_cast<int *>(static_cast<char *>(ws) + p.ws_bytes - p.order_bytes);
                launch_attn_order(a, p.nrt, C::RT, TK, p.order_shift, order, st);
            }
        }
        k_attn<T, D, WM, WK, TK, WPE, MODE>
            <<<dim3(static_cast<unsigned>(p.groups)), C::THREADS, 0, st>>>(a, p, part, ml, order);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || p.nsplit == 1)
            return e;
        if (p.nsplit < 8)
            join<T, D, 1>(a, p.nsplit, part, ml, st);
        else
            join<T, D, 8>(a, p.nsplit, part, ml, st);
        return hipGetLastError();
    }
};

template <typename F>
auto by_type(const AttnArgs &a, int D, bool bf16, F f)
{
    const int64_t R = static_cast<int64_t>(a.block_len) * (a.H / a.KV);
    const bool ranged = a.score.ranged();
    if (bf16)
        return D == 64 ? by_rows<__bf16, 64>(R, ranged, f) : by_rows<__bf16, 128>(R, ranged, f);
    return D == 64 ? by_rows<float, 64>(R, ranged, f) : by_rows<float, 128>(R, ranged, f);
}

}  // namespace
}  // namespace bdssm
