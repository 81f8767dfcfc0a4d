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
//  - float32: the matrix cores, 100 to 125 TFLOP/s.
// Eight wavefronts of 32 rows, four a SIMD at headdim 64, did better than four of 64 (half the
// LDS reads, but nothing hides a wavefront's own exponentials: 1340 against 1020 us on the
// prompt), than a third stage, 128-key tiles or a scheduled overlap inside a wavefront (no
// difference, or registers spilled).
#include <limits.h>

#include <algorithm>
#include <cmath>

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

// An infinity or a NaN among the values of a key that some rows of a workgroup attend to reaches
// its other rows through the matrix product, 0 x infinity being NaN. Where a workgroup's sums came
// out so and such a key holds such a value, its rows are computed again here, one by one and without
// the matrix cores, each from the keys that it attends to and no others. Returns whether it was so.
// (Looking through the values of tiles that rows see in part, before use, cost 2 to 6 % of every
// call; this costs nothing measurable until it is needed, and much then: a NaN among the last
// values of a prompt of 8,192 tokens on 8,192, 1.1 ms to 196 ms, which is one workgroup's 256 rows.)
template <typename T, int D>
__device__ __forceinline__ bool repair(const AttnArgs &a, const RowRange &in_lds, int *found, float *part, float2 *part_ml)
{
    const RowRange x = in_lds;
    constexpr int EL = sizeof(T), ROWB = D * EL, PPR = ROWB / 16, PL = D / 64;  // PL: channels of a lane
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, G = static_cast<int>(a.by_group.d);
    const AttnStream s = attn_stream(a, x.b);
    const int end = s.len + (a.k ? s.n : 0), page = 1 << a.page_shift;
    auto hi_of = [&](int p) {
        if (a.block == 0)
            return end;
        const int64_t h = static_cast<int64_t>(a.by_block(p) + 1) * a.block;
        return h < end ? static_cast<int>(h) : end;
    };
    auto lo_of = [&](int p) { return a.window == 0 || p < a.window ? 0 : p - a.window + 1; };
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
    const int pmin = s.len + a.by_group(x.r_first), pmax = s.len + a.by_group(x.r_end - 1);
    look(lo_of(pmin), lo_of(pmax));
    look(hi_of(pmin), hi_of(pmax));
    const int mine = __ballot(sum != sum) != 0;
    if (lane == 0)
        found[w] = mine;
    __syncthreads();
    int any = 0;
    for (int i = 0; i < x.nwaves; ++i)
        any |= found[i];
    if (!__builtin_amdgcn_readfirstlane(any))
        return false;
    const float sc = a.scale * kLog2e;
    for (int row = x.r_first + w; row < x.r_end; row += x.nwaves) {
        const int tok = a.by_group(row), head = x.kvh * G + row - tok * G, p = s.len + tok, hi = hi_of(p), lo = lo_of(p);
        const T *q = static_cast<const T *>(a.q) + (s.row0 + tok) * a.q_stride + static_cast<int64_t>(head) * D;
        float m = -__builtin_inff(), l = 0.f, o[PL] = {};
        for (int t = x.t0; t < x.t1; ++t) {
            const bool cached = t < x.ns + x.nw;
            const int first = t < x.ns ? t * x.tk : cached ? (x.w0 + t - x.ns) * x.tk : s.len + (x.c0 + t - x.ns - x.nw) * x.tk;
            const int stop = cached ? s.len : end;
            for (int kk = 0; kk < x.tk; kk += 64) {
                const int j = first + kk + lane;
                const T *k = nullptr, *v = nullptr;
                if (kk + lane < x.tk && j < stop && j < hi && (j >= lo || j < a.sinks)) {
                    k = row_of(j, a.kp, a.k, a.k_stride);
                    v = row_of(j, a.vp, a.v, a.v_stride);
                }
                float sj = 0.f;
                if (k)
                    for (int c = 0; c < D; ++c)
                        sj = fmaf(static_cast<float>(q[c]), static_cast<float>(k[c]), sj);
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

template <typename T, int D, int WM, int WK, int TK, int WPE>
__global__ __launch_bounds__((AttnCfg<T, D, WM, WK, TK>::THREADS))
__attribute__((amdgpu_waves_per_eu(WPE, WPE))) void k_attn(AttnArgs a, AttnPlan pl, float *part, float2 *part_ml)
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
    constexpr uint64_t kAll = TK < 64 ? 0xffffffffull : ~0ull;  // a mask of keys with all of them
    static_assert(C::TILE_BYTES % (1024 * NW) == 0 && TK % (32 * WK) == 0, "tile shape");

    // one array per stage and operand, so that reads of one need not wait for copies into another
    __shared__ __attribute__((aligned(16))) char k0[C::TILE_BYTES], v0[C::TILE_BYTES], k1[C::TILE_BYTES], v1[C::TILE_BYTES];
    __shared__ float2 ml[WK > 1 ? NW * 32 : 1];
    __shared__ int odd[2][NW];  // what a wavefront found, and this workgroup's part: see repair
    __shared__ RowRange mine;
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
    const int rt = a.block ? pl.nrt - 1 - rt_up : rt_up;  // ordered: the longest ranges first
    const int uk = pl.by_kv(u), kvh = pl.by_kv.rest(u), b = pl.by_split(uk), split = pl.by_split.rest(uk);
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
    auto hi_of = [&](int p) {  // keys below this are in p's block or before it
        if (a.block == 0)
            return end;
        const int64_t h = static_cast<int64_t>(a.by_block(p) + 1) * a.block;
        return h < end ? static_cast<int>(h) : end;
    };
    auto lo_of = [&](int p) { return a.window == 0 || p < a.window ? 0 : p - a.window + 1; };
    const int pmin = s.len + a.by_group(r_first), pmax = s.len + a.by_group(r_end - 1);
    const int lo_min = lo_of(pmin), lo_max = lo_of(pmax), hi_min = hi_of(pmin), hi_max = hi_of(pmax);
    const int wr0 = r_first + wm * 32;
    const bool active = wr0 < r_end;
    const int wr1 = wr0 + 31 < r_end ? wr0 + 31 : r_end - 1;
    const int w_pmin = s.len + a.by_group(wr0), w_pmax = s.len + a.by_group(wr1);
    const int w_himin = hi_of(w_pmin), w_himax = hi_of(w_pmax), w_lomax = lo_of(w_pmax), w_lomin = lo_of(w_pmin);

    // ---- tiles: sinks outside the window, the cached window, the chunk's own keys
    const int sink_len = a.window ? (a.sinks < s.len ? a.sinks : s.len) : 0;
    const int len_tiles = (s.len + TK - 1) / TK, w0 = lo_min < s.len ? lo_min / TK : len_tiles, nw = len_tiles - w0;
    const int sink_tiles = (sink_len + TK - 1) / TK, ns = sink_tiles < w0 ? sink_tiles : w0;
    const int c_lo = a.sinks > s.len || lo_min <= s.len ? 0 : lo_min - s.len, c_hi = hi_max - s.len;  // c_hi may be <= c_lo
    const int c0 = c_lo / TK, nc = n > 0 && c_hi > c_lo ? (c_hi + TK - 1) / TK - c0 : 0;
    const int nt = ns + nw + nc;
    const int per = pl.by_split(nt + nsplit - 1), t0 = split * per, t1 = t0 + per < nt ? t0 + per : nt;

    if ((lo_min != lo_max || hi_min != hi_max) && threadIdx.x == 0)
        mine = RowRange{b, kvh, split, nsplit, r_first, r_end, t0, t1, ns, nw, w0, c0, TK, NW};

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
        if (x.cached && x.start + TK <= s.len && x.start >= lo_min && whole_pages == ~0ull) {
#pragma unroll
            for (int i = 0; i < PIDS; ++i)
                valid[S.value][i] = kAll;
        } else {
#pragma unroll
            for (int i = 0; i < PIDS; ++i) {
                const int kk = 64 * i + lane, j = jpos[S.value] + kk;
                const bool there = x.cached ? (j < s.len) & ((held >> ((j >> a.page_shift) & 63)) & 1) : j < end;
                valid[S.value][i] = __ballot((kk < TK) & there & (j < hi_max) & ((j >= lo_min) | (j < a.sinks)));
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
    const int p_hi = hi_of(s.len + tok), p_lo = lo_of(s.len + tok);  // attends to [p_lo, p_hi) and below a.sinks
    const T *q_row = static_cast<const T *>(a.q) + (s.row0 + tok) * a.q_stride + static_cast<int64_t>(head) * D;
#pragma unroll
    for (int st = 0; st < L::STEPS; ++st)
        q[st] = *reinterpret_cast<const Frag *>(q_row + (2 * st + hf) * (16 / EL));

    f32x16 o[D / 32] = {};
    float m = -__builtin_inff(), l = 0.f;
    const float sc = a.scale * kLog2e;

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
    auto scores = [&](auto S) {  // S^T = K Q^T
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            sv[kb] = f32x16{};
#pragma unroll
            for (int st = 0; st < L::STEPS; ++st)
                sv[kb] = L::qk(*reinterpret_cast<const Frag *>(&KBUF(S)[koff[st] + 32 * kb * ROWB]), q[st], sv[kb]);
        }
    };
    auto hide = [&](auto S) {  // scores of what the query does not attend to: -infinity
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int blk = wk * KB + kb, jb = jpos[S.value] + 32 * blk;
            const uint32_t bits = static_cast<uint32_t>((blk < 2 ? valid[S.value][0] : valid[S.value][PIDS - 1]) >> (32 * (blk & 1)));
            // the block's keys that the query attends to, from the lane's first on
            const uint32_t see = (bits & below(p_hi - jb) & (~below(p_lo - jb) | below(a.sinks - jb))) >> (4 * hf);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const uint32_t on = __builtin_amdgcn_sbfe(see, 8 * (r / 4) + r % 4, 1);  // all bits or none
                sv[kb][r] = __uint_as_float((__float_as_uint(sv[kb][r]) & on) | (0xff800000u & ~on));
            }
        }
    };
    // the query's new reference (a lane holds half of its keys; the other half's lane has the rest)
    auto raise = [&]() {
        float mx = sv[0][0];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                mx = fmaxf(mx, sv[kb][r]);
        mx = half_max(mx) * sc;
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
    auto weigh = [&](auto S) {
        constexpr int PARTS = 2 * KB;
        const float ref = m == -__builtin_inff() ? 0.f : m;
        float wt[PARTS][8];
        bf16x8 wb[PARTS];
#pragma unroll
        for (int x = 0; x <= PARTS; ++x) {
            if (x < PARTS) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    wt[x][e] = __builtin_amdgcn_exp2f(fmaf(sv[x / 2][8 * (x % 2) + e], sc, -ref));
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
            }
            if (x > 0) {
                const int row = 16 * (x - 1);
                if constexpr (EL == 2) {
#pragma unroll
                    for (int d = 0; d < D / 32; ++d) {
                        const bf16x8 vf = cat(tr_read(reinterpret_cast<const __bf16 *>(&VBUF(S)[voff[d] + row * ROWB])),
                                              tr_read(reinterpret_cast<const __bf16 *>(&VBUF(S)[voff[d] + (row + 8) * ROWB])));
                        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, wb[x - 1], o[d], 0, 0, 0);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int d = 0; d < D / 32; ++d) {
                            const int at = voff[0] + (row + 8 * (e / 4) + e % 4) * ROWB + 128 * d;
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(*reinterpret_cast<const float *>(&VBUF(S)[at]),
                                                                        wt[x - 1][e], o[d], 0, 0, 0);
                        }
                }
            }
        }
    };

    // whether this wavefront has anything to do in the tile of stage S, and whether its rows see it whole
    auto seen = [&](auto S) {
        const int j0 = jpos[S.value];
        return active && j0 < w_himax && (j0 + TK > w_lomin || j0 < a.sinks);
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
        return full(S) && j0 + TK <= w_himin && (j0 >= w_lomax || j0 + TK <= a.sinks);
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
            if (!whole(S))
                hide(S);
            raise();
            weigh(S);
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
    if (lo_min != lo_max || hi_min != hi_max) {
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
            if (repair<T, D>(*args, mine, odd[1], part, part_ml))
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
//         of headdim 128 12.1, 15.6 so, on 16,384 keys the same
//  f32    up to 32 rows of headdim 64: 1 x 4 (32 rows, 8 streams of 4,096: 28 us, 32 us as 2 x 2,
//         47 us as 4 x 1); up to 64 rows: 2 x 2 (64 rows: 34 us, 49 us as 4 x 1; headdim 128:
//         58 us, 83 us); more: 4 x 1, whose products leave no room for more wavefronts
template <typename T, int D, typename F>
auto by_rows(int64_t R, F f)
{
    if constexpr (sizeof(T) == 2) {
        if (R <= 64)
            return f.template operator()<T, D, 2, 2, 64, (D == 64 ? 3 : 2)>();
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
    int64_t candidates(int64_t tiles) const  // 1 to so many ranges come into question
    {
        return std::max<int64_t>(1, std::min({static_cast<int64_t>(kMostRanges), f32 ? tiles : (tiles + 1) / 2,
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
        p.ws_bytes = ns > 1 ? bytes(ns) : 0;
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
        return most > 1 ? bytes(most) : 0;
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

struct Launch {
    const AttnArgs &a;
    const AttnPlan &p;
    void *ws;
    hipStream_t st;
    template <typename T, int D, int WM, int WK, int TK, int WPE>
    hipError_t operator()() const
    {
        using C = AttnCfg<T, D, WM, WK, TK>;
        float2 *ml = static_cast<float2 *>(ws);
        float *part = reinterpret_cast<float *>(static_cast<char *>(ws) + p.ml_bytes);
        k_attn<T, D, WM, WK, TK, WPE>
            <<<dim3(static_cast<unsigned>(p.groups)), C::THREADS, 0, st>>>(a, p, part, ml);
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
auto by_type(int D, bool bf16, int64_t R, F f)
{
    if (bf16)
        return D == 64 ? by_rows<__bf16, 64>(R, f) : by_rows<__bf16, 128>(R, f);
    return D == 64 ? by_rows<float, 64>(R, f) : by_rows<float, 128>(R, f);
}

}  // namespace

AttnPlan attn_plan(const AttnArgs &a, int D, bool bf16)
{
    return by_type(D, bf16, static_cast<int64_t>(a.block_len) * (a.H / a.KV), PlanOf{a});
}

size_t attn_workspace(const AttnArgs &a, int D, bool bf16)
{
    return by_type(D, bf16, static_cast<int64_t>(a.block_len) * (a.H / a.KV), WorkspaceOf{a});
}

hipError_t launch_attn(const AttnArgs &a, int D, bool bf16, const AttnPlan &p, void *ws, hipStream_t st)
{
    return by_type(D, bf16, static_cast<int64_t>(a.block_len) * (a.H / a.KV), Launch{a, p, ws, st});
}

}  // namespace bdssm
