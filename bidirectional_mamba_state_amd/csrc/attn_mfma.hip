// Attention of a chunk over a paged cache on the matrix cores (gfx950): one pass over the keys
// with a running softmax, for both element types.
//
// Work split. The query heads of one KV head are packed with the tokens into rows, row
// r = token * G + head-in-group, so that a tile of keys and values is read once for all of
// them. A workgroup owns one (stream, KV head), a tile of RT = 32 QT WM rows and a range of the
// keys that those rows attend to; a wavefront owns 32 QT rows and, where few rows leave
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
// The reference m of a query is raised, and its sums rescaled, only when a tile's maximum
// exceeds it by more than 8: weights then stay below 2^8, which float32 sums and bf16 weights
// hold as well as weights below 1.
//
// Copies. Keys and values go from the pages (or the chunk's rows) straight into LDS, 1 KB a
// copy, each copy inside one page (a page holds 16 tokens or more, a copy 8 at most); the
// 16-byte pieces of a row are permuted on the way (swz_k, swz_v) so that the operand reads are
// free of bank conflicts. Two stages: the next tile is in flight while one is computed.
//
// Masks. Per tile a 64-bit mask says which keys exist, are held and are attended to by any row
// of the workgroup; the values of the others (which may hold anything, NaN included) are cleared
// in LDS before use. Scores are selected per element in tiles that some row of a wavefront does
// not see whole; the other tiles skip that.
#include <algorithm>
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
constexpr float kRaise = 8.f;  // see "Softmax" above

#define kOnes (bf16x2{static_cast<__bf16>(1.f), static_cast<__bf16>(1.f)})

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

// the n lowest bits, for any n
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

template <int N>
struct Int {
    static constexpr int value = N;
};

template <typename T, int D, int QT, int WM, int WK, int TK>
struct AttnCfg {
    static constexpr int NW = WM * WK, THREADS = 64 * NW, RT = 32 * QT * WM;
    static constexpr int TILE_BYTES = TK * Tile<T, D>::ROWB;
};

template <typename T, int D, int QT, int WM, int WK, int TK, int WPE>
__global__ __launch_bounds__((AttnCfg<T, D, QT, WM, WK, TK>::THREADS))
__attribute__((amdgpu_waves_per_eu(WPE, WPE))) void k_attn(AttnArgs a, AttnPlan pl, float *part, float2 *part_ml)
{
    using C = AttnCfg<T, D, QT, WM, WK, TK>;
    using L = Tile<T, D>;
    using Frag = typename L::Frag;
    constexpr int NW = C::NW, ROWB = L::ROWB, PPR = ROWB / 16;
    constexpr int RPC = 1024 / ROWB;                // rows of a copy
    constexpr int NC = C::TILE_BYTES / 1024 / NW;   // copies of a wavefront per tile, of K and of V
    constexpr int PIDS = (TK + 63) / 64;            // page number registers of a tile
    constexpr int KB = TK / 32 / WK;                // 32-key blocks of a wavefront per tile,
    constexpr int KS = KB < 2 ? KB : 2;             // KS of them per softmax step
    constexpr int EL = sizeof(T);
    static_assert(C::TILE_BYTES % (1024 * NW) == 0 && TK % (32 * WK) == 0 , "tile shape");

    // one array per stage and operand, so that reads of one need not wait for copies into another
    __shared__ __attribute__((aligned(16))) char k0[C::TILE_BYTES], v0[C::TILE_BYTES], k1[C::TILE_BYTES], v1[C::TILE_BYTES];
    __shared__ float2 ml[WK > 1 ? NW * QT * 32 : 1];
    auto KBUF = [&](auto S) -> char * { return S.value == 0 ? k0 : k1; };
    auto VBUF = [&](auto S) -> char * { return S.value == 0 ? v0 : v1; };

    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / WK, wk = w % WK, hf = lane >> 5, l32 = lane & 31;

    // ---- this workgroup's part, row tile and unit (see AttnPlan)
    const int nsplit = pl.nsplit, wid = blockIdx.x >> 3;
    const int part_no = (pl.rt_fast ? wid / pl.nrt_sub : wid % pl.per_xcd) * 8 + (blockIdx.x & 7);
    if (part_no >= pl.units)
        return;
    const int per_sub = pl.units / pl.sub, u = part_no % per_sub;
    const int rt_up = (pl.rt_fast ? wid % pl.nrt_sub : wid / pl.per_xcd) * pl.sub + part_no / per_sub;
    if (rt_up >= pl.nrt)
        return;
    const int rt = a.block ? pl.nrt - 1 - rt_up : rt_up;  // ordered: the longest ranges first
    const int kvh = u % a.KV, split = u / a.KV % nsplit, b = u / a.KV / nsplit, G = a.H / a.KV;
    const AttnStream s = attn_stream(a, b);
    const int rows = s.n * G, r_first = rt * C::RT;
    if (r_first >= rows)
        return;

    // ---- what the workgroup's rows and this wavefront's rows attend to
    const int n = a.k ? s.n : 0, end = s.len + n;  // keys at positions [0, end)
    auto hi_of = [&](int p) {  // keys below this are in p's block or before it
        if (a.block == 0)
            return end;
        const int64_t h = static_cast<int64_t>(p / a.block + 1) * a.block;
        return h < end ? static_cast<int>(h) : end;
    };
    auto lo_of = [&](int p) { return a.window == 0 || p < a.window ? 0 : p - a.window + 1; };
    const int r_last = (r_first + C::RT < rows ? r_first + C::RT : rows) - 1;
    const int lo_min = lo_of(s.len + r_first / G), hi_max = hi_of(s.len + r_last / G);
    const int wr0 = r_first + wm * 32 * QT;
    const bool active = wr0 < rows;
    const int wr1 = wr0 + 32 * QT - 1 < rows ? wr0 + 32 * QT - 1 : rows - 1;
    const int w_pmin = s.len + wr0 / G, w_pmax = s.len + wr1 / G;
    const int w_himin = hi_of(w_pmin), w_himax = hi_of(w_pmax), w_lomax = lo_of(w_pmax), w_lomin = lo_of(w_pmin);

    // ---- tiles: sinks outside the window, the cached window, the chunk's own keys
    const int sink_len = a.window ? (a.sinks < s.len ? a.sinks : s.len) : 0;
    const int len_tiles = (s.len + TK - 1) / TK, w0 = lo_min < s.len ? lo_min / TK : len_tiles, nw = len_tiles - w0;
    const int sink_tiles = (sink_len + TK - 1) / TK, ns = sink_tiles < w0 ? sink_tiles : w0;
    const int c_lo = a.sinks > s.len || lo_min <= s.len ? 0 : lo_min - s.len, c_hi = hi_max - s.len;  // c_hi may be <= c_lo
    const int c0 = c_lo / TK, nc = n > 0 && c_hi > c_lo ? (c_hi + TK - 1) / TK - c0 : 0;
    const int nt = ns + nw + nc;
    const int per = (nt + nsplit - 1) / nsplit, t0 = split * per, t1 = t0 + per < nt ? t0 + per : nt;

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
    const int *table = a.table + static_cast<int64_t>(b) * a.max_pages;
    const int page = 1 << a.page_shift, last_page = (s.len > 0 ? s.len - 1 : 0) >> a.page_shift;
    // Page numbers: lane i holds the one of page pbase + i (pbase a multiple of 64, so that no
    // tile straddles it), and in `ids_next` the one of 64 pages on.
    int pbase = -1, ids = 0, ids_next = 0;
    uint64_t held = 0;  // which of the 64 are pages of the pool
    auto page_no = [&](int i) { return table[i < last_page ? i : last_page]; };
    auto find_pages = [&](int start) {
        const int p = (start >> a.page_shift) & ~63;
        if (p != pbase) {
            ids = pbase >= 0 && p == pbase + 64 ? ids_next : page_no(p + lane);
            ids_next = page_no(p + 64 + lane);
            pbase = p;
            held = __ballot(static_cast<uint32_t>(ids) < static_cast<uint32_t>(a.num_pages));
        }
    };
    const int crow = lane / PPR, cslot = lane % PPR;  // row of a copy, LDS piece of that row
    const int page_bytes = page * ROWB;
    const uint32_t pool_step = static_cast<uint32_t>(a.KV * page_bytes);  // from page to page
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
#pragma unroll
        for (int i = 0; i < PIDS; ++i) {
            const int kk = 64 * i + lane, j = jpos[S.value] + kk;
            const bool there = x.cached ? (j < s.len) & ((held >> ((j >> a.page_shift) & 63)) & 1) : j < end;
            valid[S.value][i] = __ballot((kk < TK) & there & (j < hi_max) & ((j >= lo_min) | (j < a.sinks)));
        }
        if (x.cached) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int row0 = (w + NW * c) * RPC, row = row0 + crow;
                const int pi = ((x.start + row0) >> a.page_shift) & 63;
                const uint32_t pg = __builtin_amdgcn_readlane(ids, pi);
                const bool ok = (held >> pi) & 1;  // not held: an empty range, nothing is read
                const uint64_t base = ok ? static_cast<uint64_t>(pg) * pool_step : 0;
                const int off = ((x.start + row0) & (page - 1)) * ROWB + crow * ROWB;
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
    Frag q[QT][L::STEPS];
    int p_hi[QT], p_lo[QT];  // the lane's query attends to keys in [p_lo, p_hi) and below a.sinks
#pragma unroll
    for (int i = 0; i < QT; ++i) {
        int r = wr0 + 32 * i + l32;
        r = r < rows ? r : rows - 1;
        const int tok = r / G, head = kvh * G + r % G;
        p_hi[i] = hi_of(s.len + tok), p_lo[i] = lo_of(s.len + tok);
        const T *qr = static_cast<const T *>(a.q) + (s.row0 + tok) * a.q_stride + static_cast<int64_t>(head) * D;
#pragma unroll
        for (int st = 0; st < L::STEPS; ++st)
            q[i][st] = *reinterpret_cast<const Frag *>(qr + (2 * st + hf) * (16 / EL));
    }

    f32x16 o[QT][D / 32] = {};
    float m[QT], l[QT];
#pragma unroll
    for (int i = 0; i < QT; ++i)
        m[i] = -__builtin_inff(), l[i] = 0.f;
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

    // ---- a step: KS blocks of 32 keys of a tile, from this wavefront's block B0 on
    f32x16 sv[KS][QT];                                                         // scores
    typename std::conditional<EL == 2, bf16x8[2 * KS][QT], f32x16[KS][QT]>::type pw;  // weights, B operands
    auto scores = [&](auto S, auto B0) {  // S^T = K Q^T
#pragma unroll
        for (int kb = 0; kb < KS; ++kb) {
#pragma unroll
            for (int i = 0; i < QT; ++i)
                sv[kb][i] = f32x16{};
#pragma unroll
            for (int st = 0; st < L::STEPS; ++st) {
                const Frag kf = *reinterpret_cast<const Frag *>(&KBUF(S)[koff[st] + 32 * (B0.value + kb) * ROWB]);
#pragma unroll
                for (int i = 0; i < QT; ++i)
                    sv[kb][i] = L::qk(kf, q[i][st], sv[kb][i]);
            }
        }
    };
    // the lane's queries over their keys (half of them; the other half's lane has the rest)
    auto softmax = [&](auto S, auto B0, bool whole) {
        if (!whole) {
#pragma unroll
            for (int kb = 0; kb < KS; ++kb) {
                const int blk = wk * KB + B0.value + kb, jb = jpos[S.value] + 32 * blk;
                const uint32_t bits = static_cast<uint32_t>((blk < 2 ? valid[S.value][0] : valid[S.value][PIDS - 1]) >> (32 * (blk & 1)));
                const uint32_t sink = below(a.sinks - jb);
#pragma unroll
                for (int i = 0; i < QT; ++i) {
                    // the block's keys that the lane's query attends to, from the lane's first on
                    const uint32_t see = (bits & below(p_hi[i] - jb) & (~below(p_lo[i] - jb) | sink)) >> (4 * hf);
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const uint32_t on = __builtin_amdgcn_sbfe(see, 8 * (r / 4) + r % 4, 1);  // all bits or none
                        sv[kb][i][r] = __uint_as_float((__float_as_uint(sv[kb][i][r]) & on) | (0xff800000u & ~on));
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < QT; ++i) {
            float mx = sv[0][i][0];
#pragma unroll
            for (int kb = 0; kb < KS; ++kb)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    mx = fmaxf(mx, sv[kb][i][r]);
            mx = half_max(mx) * sc;
            if (__ballot(mx > m[i] + kRaise)) {
                const float mn = fmaxf(m[i], mx);
                const float f = m[i] == mn ? 1.f : __builtin_amdgcn_exp2f(m[i] - mn);  // equal infinities: 1
                m[i] = mn;
                l[i] *= f;
#pragma unroll
                for (int d = 0; d < D / 32; ++d)
                    o[i][d] *= f;
            }
            const float ref = m[i] == -__builtin_inff() ? 0.f : m[i];
#pragma unroll
            for (int kb = 0; kb < KS; ++kb) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] = __builtin_amdgcn_exp2f(fmaf(sv[kb][i][8 * x + e], sc, -ref));
                    if constexpr (EL == 2) {
                        const bf16x8 h = to_bf16x8(f);
                        pw[2 * kb + x][i] = h;
                        // the sum is of the rounded weights, two per instruction
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            l[i] = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{h[2 * e], h[2 * e + 1]}, kOnes, l[i], false);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            pw[kb][i][8 * x + e] = f[e];
                            l[i] += f[e];
                        }
                    }
                }
            }
        }
    };
    auto values = [&](auto S, auto B0) {  // O^T += V^T P^T
#pragma unroll
        for (int kb = 0; kb < KS; ++kb) {
            const int row = 32 * (B0.value + kb);
            if constexpr (EL == 2) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int d = 0; d < D / 32; ++d) {
                        const bf16x8 vf =
                            cat(tr_read(reinterpret_cast<const __bf16 *>(&VBUF(S)[voff[d] + (row + 16 * x) * ROWB])),
                                tr_read(reinterpret_cast<const __bf16 *>(&VBUF(S)[voff[d] + (row + 16 * x + 8) * ROWB])));
#pragma unroll
                        for (int i = 0; i < QT; ++i)
                            o[i][d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pw[2 * kb + x][i], o[i][d], 0, 0, 0);
                    }
            } else {
#pragma unroll
                for (int r = 0; r < 16; ++r)
#pragma unroll
                    for (int d = 0; d < D / 32; ++d) {
                        const float vf = *reinterpret_cast<const float *>(
                            &VBUF(S)[voff[0] + (row + 8 * (r / 4) + r % 4) * ROWB + 128 * d]);
#pragma unroll
                        for (int i = 0; i < QT; ++i)
                            o[i][d] = __builtin_amdgcn_mfma_f32_32x32x2f32(vf, pw[kb][i][r], o[i][d], 0, 0, 0);
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
            all = all && valid[S.value][i] == (TK < 64 ? 0xffffffffull : ~0ull);
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
    for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int st = 0; st < L::STEPS; ++st)
            asm volatile("" : "+v"(q[i][st]));

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
            const bool wh = whole(S);
            scores(S, Int<0>{});
            softmax(S, Int<0>{}, wh);
            values(S, Int<0>{});
            if constexpr (KB > KS) {
                scores(S, Int<KS>{});
                softmax(S, Int<KS>{}, wh);
                values(S, Int<KS>{});
            }
        }
    };
    if (t0 < t1)
        start(Int<0>{});
    for (int t = t0; t < t1; t += 2) {
        step(Int<0>{}, t);
        if (t + 1 < t1)
            step(Int<1>{}, t + 1);
    }
#pragma unroll
    for (int i = 0; i < QT; ++i)
        l[i] = half_sum(l[i]);

    // ---- wavefronts that shared the rows: join in LDS, in wavefront order
    if constexpr (WK > 1) {
        constexpr int UNIT = 32 * D * 4, PER = C::TILE_BYTES / UNIT;  // bytes of 32 rows; units per array
        static_assert((WK - 1) * WM * QT <= 4 * PER, "the stages hold the partial rows");
        auto unit = [&](int u) -> float * {
            char *arr = u / PER == 0 ? k0 : u / PER == 1 ? v0 : u / PER == 2 ? k1 : v1;
            return reinterpret_cast<float *>(arr + (u % PER) * UNIT);
        };
        __syncthreads();
#pragma unroll
        for (int i = 0; i < QT; ++i) {
            if (hf == 0)
                ml[(w * QT + i) * 32 + l32] = make_float2(m[i], l[i]);
            if (wk > 0) {
                f32x4 *u = reinterpret_cast<f32x4 *>(unit(((wk - 1) * WM + wm) * QT + i));
#pragma unroll
                for (int d = 0; d < D / 32; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        u[(d * 4 + r) * 64 + lane] = f32x4{o[i][d][4 * r], o[i][d][4 * r + 1], o[i][d][4 * r + 2], o[i][d][4 * r + 3]};
            }
        }
        __syncthreads();
        if (wk > 0)
            return;
#pragma unroll
        for (int i = 0; i < QT; ++i) {
            float mt = m[i];
#pragma unroll
            for (int x = 1; x < WK; ++x)
                mt = fmaxf(mt, ml[((w + x) * QT + i) * 32 + l32].x);
            const float f0 = m[i] == mt ? 1.f : __builtin_amdgcn_exp2f(m[i] - mt);
            l[i] *= f0;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
                o[i][d] *= f0;
#pragma unroll
            for (int x = 1; x < WK; ++x) {
                const float2 om = ml[((w + x) * QT + i) * 32 + l32];
                const float f = om.x == mt ? 1.f : __builtin_amdgcn_exp2f(om.x - mt);
                l[i] = fmaf(om.y, f, l[i]);
                const f32x4 *u = reinterpret_cast<const f32x4 *>(unit(((x - 1) * WM + wm) * QT + i));
#pragma unroll
                for (int d = 0; d < D / 32; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const f32x4 ov = u[(d * 4 + r) * 64 + lane];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[i][d][4 * r + e] = fmaf(ov[e], f, o[i][d][4 * r + e]);
                    }
            }
            m[i] = mt;
        }
    }

    // ---- rows out: normalized, or partial with their maximum and sum
    const int64_t R = static_cast<int64_t>(a.block_len) * G;
#pragma unroll
    for (int i = 0; i < QT; ++i) {
        const int r = wr0 + 32 * i + l32;
        if (r >= rows)
            continue;
        if (nsplit == 1) {
            const float inv = l[i] > 0.f ? 1.f / l[i] : l[i];  // nothing attended to: 0; NaN stays
            T *out = static_cast<T *>(a.out) + ((s.row0 + r / G) * a.H + kvh * G + r % G) * D + 4 * hf;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const f32x4 ov = f32x4{o[i][d][4 * x], o[i][d][4 * x + 1], o[i][d][4 * x + 2], o[i][d][4 * x + 3]} * inv;
                    if constexpr (EL == 2)
                        *reinterpret_cast<bf16x4 *>(out + 32 * d + 8 * x) = __builtin_convertvector(ov, bf16x4);
                    else
                        *reinterpret_cast<f32x4 *>(out + 32 * d + 8 * x) = ov;
                }
        } else {
            const int64_t u = ((static_cast<int64_t>(b) * a.KV + kvh) * nsplit + split) * R + r;
            if (hf == 0)
                part_ml[u] = make_float2(m[i], l[i]);
            float *out = part + u * D + 4 * hf;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    *reinterpret_cast<f32x4 *>(out + 32 * d + 8 * x) =
                        f32x4{o[i][d][4 * x], o[i][d][4 * x + 1], o[i][d][4 * x + 2], o[i][d][4 * x + 3]};
        }
    }
}

// Joins the partial rows of a split cache: out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,
// in split order. D/4 lanes hold a row; a split whose range was empty (sum 0) is not read.
template <typename T, int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, int nsplit, const float *part, const float2 *part_ml)
{
    constexpr int LPR = D / 4;
    const int b = blockIdx.z, kvh = blockIdx.y, G = a.H / a.KV;
    const int r = blockIdx.x * (256 / LPR) + threadIdx.x / LPR, c = 4 * (threadIdx.x % LPR);
    const AttnStream s = attn_stream(a, b);
    if (r >= s.n * G)
        return;
    const int64_t R = static_cast<int64_t>(a.block_len) * G, u0 = (static_cast<int64_t>(b) * a.KV + kvh) * nsplit * R + r;
    float M = -__builtin_inff();
    for (int x = 0; x < nsplit; ++x)
        M = fmaxf(M, part_ml[u0 + x * R].x);
    float l = 0.f;
    f32x4 o = {};
#pragma unroll 4
    for (int x = 0; x < nsplit; ++x) {
        const float2 v = part_ml[u0 + x * R];
        const f32x4 ov = *reinterpret_cast<const f32x4 *>(part + (u0 + x * R) * D + c);
        const float f = v.x == M ? 1.f : __builtin_amdgcn_exp2f(v.x - M);
        l = fmaf(v.y, f, l);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = fmaf(ov[e], f, o[e]);
    }
    const float inv = l > 0.f ? 1.f / l : l;
    o *= inv;
    T *out = static_cast<T *>(a.out) + ((s.row0 + r / G) * a.H + kvh * G + r % G) * D + c;
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<bf16x4 *>(out) = __builtin_convertvector(o, bf16x4);
    else
        *reinterpret_cast<f32x4 *>(out) = o;
}

// f(QT, WM, WK, TK, WPE): the kernel shape for R rows per (stream, KV head).
template <typename T, int D, typename F>
auto by_rows(int64_t R, F f)
{
    if constexpr (sizeof(T) == 2) {
        if (R <= 32)
            return f.template operator()<T, D, 1, 1, 4, 128, 1>();
        if (R <= 64)
            return f.template operator()<T, D, 2, 1, 4, 128, 1>();
        if (R <= 128)
            return f.template operator()<T, D, 2, 2, 2, 64, (D == 64 ? 2 : 1)>();
        return f.template operator()<T, D, 1, 8, 1, 64, (D == 64 ? 4 : 2)>();
    } else {
        if (R <= 32)
            return f.template operator()<T, D, 1, 1, (D == 64 ? 4 : 2), (D == 64 ? 128 : 64), 1>();
        return f.template operator()<T, D, 1, 4, 1, (D == 64 ? 64 : 32), 2>();
    }
}

struct PlanOf {
    const AttnArgs &a;
    template <typename T, int D, int QT, int WM, int WK, int TK, int WPE>
    AttnPlan operator()() const
    {
        using C = AttnCfg<T, D, QT, WM, WK, TK>;
        AttnPlan p{};
        const int64_t R = static_cast<int64_t>(a.block_len) * (a.H / a.KV);
        p.nrt = static_cast<int>((R + C::RT - 1) / C::RT);
        // Ranges: the number whose rounds of workgroups take the fewest tiles in all, where a
        // workgroup costs about six tiles beside its own, and a join about six more.
        const int64_t vis = a.window && static_cast<int64_t>(a.window) + a.block_len < a.max_len
                                ? static_cast<int64_t>(a.window) + a.block_len + a.sinks
                                : a.max_len;
        const int64_t tiles = (vis + a.block_len + TK - 1) / TK, units = static_cast<int64_t>(a.batch) * a.KV;
        const int64_t slots = static_cast<int64_t>(device_cus()) * (4 * WPE / C::NW);
        int64_t ns = 1, best = INT64_MAX;
        for (int64_t x = 1; x <= 64 && x <= (tiles + 3) / 4; ++x) {
            const int64_t cost = (units * p.nrt * x + slots - 1) / slots * ((tiles + x - 1) / x + 6) + (x > 1 ? 6 : 0);
            if (cost < best)
                best = cost, ns = x;
        }
        p.nsplit = static_cast<int>(ns);
        const int64_t all = units * ns;
        p.sub = static_cast<int>(all >= 64 ? 1 : std::min<int64_t>(p.nrt, (64 + all - 1) / all));
        p.nrt_sub = (p.nrt + p.sub - 1) / p.sub;
        p.units = static_cast<int>(all * p.sub);
        p.per_xcd = (p.units + 7) / 8;
        p.rt_fast = p.nrt_sub <= 4;
        const int64_t rows = static_cast<int64_t>(a.batch) * a.KV * ns * R;
        p.ml_bytes = ns > 1 ? static_cast<size_t>((rows * 8 + 255) / 256 * 256) : 0;
        p.ws_bytes = ns > 1 ? p.ml_bytes + static_cast<size_t>(rows) * D * 4 : 0;
        return p;
    }
};

struct Launch {
    const AttnArgs &a;
    const AttnPlan &p;
    void *ws;
    hipStream_t st;
    template <typename T, int D, int QT, int WM, int WK, int TK, int WPE>
    hipError_t operator()() const
    {
        using C = AttnCfg<T, D, QT, WM, WK, TK>;
        float2 *ml = static_cast<float2 *>(ws);
        float *part = reinterpret_cast<float *>(static_cast<char *>(ws) + p.ml_bytes);
        k_attn<T, D, QT, WM, WK, TK, WPE>
            <<<dim3(static_cast<unsigned>(8 * p.per_xcd) * p.nrt_sub), C::THREADS, 0, st>>>(a, p, part, ml);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || p.nsplit == 1)
            return e;
        const int64_t R = static_cast<int64_t>(a.block_len) * (a.H / a.KV);
        k_attn_join<T, D><<<dim3(static_cast<unsigned>((R * (D / 4) + 255) / 256), a.KV, a.batch), 256, 0, st>>>(
            a, p.nsplit, part, ml);
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

hipError_t launch_attn(const AttnArgs &a, int D, bool bf16, const AttnPlan &p, void *ws, hipStream_t st)
{
    return by_type(D, bf16, static_cast<int64_t>(a.block_len) * (a.H / a.KV), Launch{a, p, ws, st});
}

}  // namespace bdssm
