// Upkeep of a paged cache: taking and giving back pages (bdssm_pages_advance), forking streams
// (bdssm_pages_fork), moving the used pages to the front (bdssm_pages_compact) and copying pages
// (bdssm_pages_copy).
//
// The first launch of each takes a snapshot of which pages are free, one bit a page, with a count per
// chunk of the pool, and counts what each stream needs. In the second every stream finds its place
// among the needs (the sum of those in front of it) and the free pages of those ranks (free_pages);
// a compaction lists them first, in a launch of its own. Nothing is handed out by an atomic counter,
// so that results depend on the contents alone; the uses of pages are counted by integer atomics,
// whose sum has no order. The snapshot lets uses_out be uses itself. Small pools: one launch, below.
#include <limits.h>

#include <algorithm>

#include "attn.h"
#include "internal.h"

namespace bdssm {
namespace {

constexpr int kWords = 64;            // words of 64 pages that a workgroup takes of the pool,
constexpr int kChunk = 64 * kWords;   // and so many pages

struct PoolArgs {
    const int *table, *lens, *uses;
    int *table_out, *uses_out;
    int batch, page_shift, num_pages, max_pages, chunks, row_parts;
    // workspace
    uint64_t *bits;  // [chunks][kWords]: the page is free
    int *counts;     // [chunks] free pages
    int *needs;      // [batch]
    int *list;       // [num_pages] compact: free pages in order
    int *map;        // [num_pages] compact: which move a page is, or -1
    int *moves;      // [1] compact: number of moves
};

// sums over a workgroup of 256 threads, in every thread; lds: 4 N
template <int N>
__device__ __forceinline__ void block_sums(int (&v)[N], int *lds)
{
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int y = 1; y < 64; y *= 2)
            v[k] += __shfl_xor(v[k], y);
    __syncthreads();  // lds may still be read from an earlier sum
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int k = 0; k < N; ++k)
            lds[4 * k + (threadIdx.x >> 6)] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k)
        v[k] = lds[4 * k] + lds[4 * k + 1] + lds[4 * k + 2] + lds[4 * k + 3];
}
__device__ __forceinline__ int block_sum(int v, int *lds)
{
    int x[1] = {v};
    block_sums(x, lds);
    return x[0];
}

// sum of v[0 .. n), by a workgroup
__device__ __forceinline__ int sum_of(const int *v, int n, int *lds)
{
    int s = 0;
    for (int i = threadIdx.x; i < n; i += 256)
        s += v[i];
    return block_sum(s, lds);
}

// A chunk of the snapshot, and uses as they go on being counted (none below 0). All of a thread's uses
// are loaded before the first is stored: in place the compiler would wait for each (5.4 us for the
// launch that has this, 3.9 so).
__device__ __forceinline__ void snapshot(const PoolArgs &a, int chunk, int *lds)
{
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t first = static_cast<int64_t>(chunk) * kChunk + 64 * w + lane;
    int u[kWords / 4], n = 0;
#pragma unroll
    for (int k = 0; k < kWords / 4; ++k) {
        const int64_t p = first + 256 * k;
        u[k] = a.uses[p < a.num_pages ? p : a.num_pages - 1];
    }
#pragma unroll
    for (int k = 0; k < kWords / 4; ++k) {
        const int64_t p = first + 256 * k;
        const uint64_t word = __ballot(p < a.num_pages && u[k] <= 0);
        if (p < a.num_pages && (u[k] < 0 || a.uses_out != a.uses))
            a.uses_out[p] = u[k] > 0 ? u[k] : 0;
        if (lane == 0)
            a.bits[static_cast<int64_t>(chunk) * kWords + w + 4 * k] = word;
        n += __popcll(word);  // the same in every lane
    }
    const int all = block_sum(lane == 0 ? n : 0, lds);
    if (threadIdx.x == 0)
        a.counts[chunk] = all;
}

__device__ __forceinline__ int cached(const PoolArgs &a, int b)
{
    const int64_t held = static_cast<int64_t>(a.max_pages) << a.page_shift;
    const int len = a.lens[b];
    return len < 0 ? 0 : len > held ? static_cast<int>(held) : len;
}

__device__ __forceinline__ bool is_page(const PoolArgs &a, int e) { return e >= 0 && e < a.num_pages; }

// ---- advance
struct AdvanceArgs {
    PoolArgs p;
    const int *starts;
    int block_len, window, sinks;
    int *lacking;
};

struct Span {
    int from, to;  // entries that a stream's new tokens start: from the first page at or past its length
    int len;
};

__device__ __forceinline__ Span new_entries(const AdvanceArgs &a, int b)
{
    const int len = cached(a.p, b), page = 1 << a.p.page_shift;
    int64_t n = a.block_len;
    if (a.starts) {
        n = static_cast<int64_t>(a.starts[b + 1]) - a.starts[b];
        n = n < 0 ? 0 : n > a.block_len ? a.block_len : n;
    }
    const int64_t held = static_cast<int64_t>(a.p.max_pages) << a.p.page_shift;
    const int64_t end = len + n < held ? len + n : held;
    return Span{static_cast<int>((static_cast<int64_t>(len) + page - 1) >> a.p.page_shift),
                static_cast<int>((end + page - 1) >> a.p.page_shift), len};
}

// What an entry that new tokens do not start is afterwards. The next query is at position len and
// looks back to len - window + 1.
__device__ __forceinline__ bool stays(const AdvanceArgs &a, const Span &s, int i, int e)
{
    const int64_t at = static_cast<int64_t>(i) << a.p.page_shift;
    return i < s.from && is_page(a.p, e) &&
           (a.window == 0 || at < a.sinks || at + (int64_t{1} << a.p.page_shift) > static_cast<int64_t>(s.len) - a.window + 1);
}

// empty entries among [from, to) of a row, by a workgroup
__device__ __forceinline__ int empty_entries(const PoolArgs &a, const int *row, int from, int to, int *lds)
{
    int n = 0;
    for (int i = from + threadIdx.x; i < to; i += 256)
        n += !is_page(a, row[i]);
    return block_sum(n, lds);
}

__global__ __launch_bounds__(256) void k_advance_count(AdvanceArgs a)
{
    __shared__ int lds[4];
    if (static_cast<int>(blockIdx.x) < a.p.chunks)
        return snapshot(a.p, blockIdx.x, lds);
    const int b = blockIdx.x - a.p.chunks;
    const Span s = new_entries(a, b);
    const int n = empty_entries(a.p, a.p.table + static_cast<int64_t>(b) * a.p.max_pages, s.from, s.to, lds);
    if (threadIdx.x == 0)
        a.p.needs[b] = n;
}

// Lane l: the free pages in front of word l of a chunk (a word a lane), after those in front of it.
__device__ __forceinline__ int words_before(uint64_t word, int before)
{
    const int own = __popcll(word);
    int n = own;
#pragma unroll
    for (int y = 1; y < 64; y *= 2) {
        const int o = __shfl_up(n, y);
        n += static_cast<int>(threadIdx.x & 63) >= y ? o : 0;
    }
    return before + n - own;
}

// The free pages of ranks [from, from + n) into LDS (n up to kTake; -1 past the last), by a workgroup:
// the chunks that hold them by a running sum of the counts (`mine`: the thread's of the first 256),
// their words by one lane each.
constexpr int kTake = 1024;

__device__ __forceinline__ void free_pages(const PoolArgs &a, int mine, int from, int n, int *out, int *lds)
{
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    __syncthreads();  // `out` may still be read
    for (int i = threadIdx.x; i < n; i += 256)
        out[i] = -1;
    for (int c0 = 0, before = 0; c0 < a.chunks && before < from + n; c0 += 256) {
        const int c = c0 + threadIdx.x, count = c0 == 0 ? mine : c < a.chunks ? a.counts[c] : 0;
        int sum = count;
#pragma unroll
        for (int y = 1; y < 64; y *= 2) {
            const int o = __shfl_up(sum, y);
            sum += lane >= y ? o : 0;
        }
        __syncthreads();
        if (lane == 63)
            lds[w] = sum;
        __syncthreads();
        int first = before + sum - count;  // rank of the chunk's first
        for (int x = 0; x < w; ++x)
            first += lds[x];
        before += lds[0] + lds[1] + lds[2] + lds[3];
        for (uint64_t hits = __ballot(count > 0 && first < from + n && first + count > from); hits; hits &= hits - 1) {
            const int l = __builtin_ctzll(hits), chunk = c0 + 64 * w + l;
            uint64_t word = a.bits[static_cast<int64_t>(chunk) * kWords + lane];
            for (int r = words_before(word, __shfl(first, l)); word && r < from + n; ++r, word &= word - 1)
                if (r >= from)
                    out[r - from] = chunk * kChunk + 64 * lane + __builtin_ctzll(word);
        }
    }
    __syncthreads();
}

// A row's part [from, to) of `parts`.
__device__ __forceinline__ Span part_of(const PoolArgs &a, int part)
{
    const int per = (a.max_pages + a.row_parts - 1) / a.row_parts;
    const int64_t from = static_cast<int64_t>(part) * per;
    return Span{static_cast<int>(from < a.max_pages ? from : a.max_pages),
                static_cast<int>(from + per < a.max_pages ? from + per : a.max_pages), 0};
}

// f(i, x[i], y[i]) for i in a part, by a workgroup; four of a thread are loaded before the first is used
template <typename F>
__device__ __forceinline__ void part_entries(const Span &part, const int *x, const int *y, F f)
{
    constexpr int U = 4;
    for (int64_t i0 = part.from + threadIdx.x; i0 < part.to; i0 += 256 * U) {
        int u[U], v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t i = i0 + 256 * k < part.to ? i0 + 256 * k : part.to - 1;
            u[k] = x[i], v[k] = y[i];
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i0 + 256 * k < part.to)
                f(static_cast<int>(i0 + 256 * k), u[k], v[k]);
    }
}

// The free pages of the pool, and what the streams in front of stream b need; for the first stream, what
// all of them need. Loaded at a kernel's start, beside what the rest of it waits for, and summed later.
struct Balance {
    int count, need;  // of this thread: chunk threadIdx.x, and stream threadIdx.x of those that count
    int free, needs;  // sums
    __device__ __forceinline__ Balance(const PoolArgs &a, int b)
        : count(static_cast<int>(threadIdx.x) < a.chunks ? a.counts[threadIdx.x] : 0),
          need(static_cast<int>(threadIdx.x) < (b == 0 ? a.batch : b) ? a.needs[threadIdx.x] : 0), free(0), needs(0)
    {
    }
    __device__ __forceinline__ void sum(const PoolArgs &a, int b, int *lds)  // lds: 8
    {
        int v[2] = {count, need};
        for (int i = 256 + threadIdx.x; i < a.chunks; i += 256)
            v[0] += a.counts[i];
        for (int i = 256 + threadIdx.x, n = b == 0 ? a.batch : b; i < n; i += 256)
            v[1] += a.needs[i];
        block_sums(v, lds);
        free = v[0], needs = v[1];
    }
};

// Rows, a part of one each: gives back, takes, counts. The entries that new tokens start are the
// first workgroup's of a row, so that none is ranked by a table that another one has begun to fill; a
// row of several parts has one more workgroup for them, since both are chains of loads
// (64 rows of 16,384 entries: 7.3 us, 6.5 so).
__global__ __launch_bounds__(256) void k_advance_rows(AdvanceArgs a)
{
    __shared__ int lds[8], list[kTake];
    const int b = blockIdx.y, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    if (b >= a.p.batch) {  // no streams
        if (threadIdx.x == 0)
            a.lacking[0] = 0;
        return;
    }
    const int64_t row = static_cast<int64_t>(b) * a.p.max_pages;
    const int *in = a.p.table + row;
    int *out = a.p.table_out + row;
    Balance all(a.p, b);
    const int own = a.p.needs[b];
    const Span s = new_entries(a, b), none{};
    const bool whole_row = gridDim.x == 1;
    part_entries(whole_row ? part_of(a.p, 0) : blockIdx.x ? part_of(a.p, blockIdx.x - 1) : none, in, in, [&](int i, int e, int) {
        if (i >= s.from && i < s.to)
            return;
        const bool kept = stays(a, s, i, e);
        if (!kept && is_page(a.p, e))
            atomicSub(&a.p.uses_out[e], 1);
        if (in != out || !kept)
            out[i] = kept ? e : -1;
    });
    if (blockIdx.x != 0 || (b != 0 && s.from >= s.to))
        return;
    auto entry = [&](int i) { return i < s.to ? in[i] : 0; };
    int next = entry(s.from + threadIdx.x);
    all.sum(a.p, b, lds);
    if (b == 0 && threadIdx.x == 0)
        a.lacking[0] = all.needs > all.free ? all.needs - all.free : 0;
    const int place = b == 0 ? 0 : all.needs;
    int taken = 0, first = 0, listed = 0;  // of the stream's needs: met, and listed [first, listed)
    for (int i0 = s.from; i0 < s.to; i0 += 256) {
        if (taken + 256 > listed && listed < own) {  // the next 256 entries may need more than are listed
            listed = taken + kTake < own ? taken + kTake : own;
            free_pages(a.p, all.count, place + taken, listed - taken, list, lds);
            first = taken;
        }
        const int i = i0 + threadIdx.x, e = next;
        next = entry(i + 256);
        const bool empty = i < s.to && !is_page(a.p, e);
        const uint64_t word = __ballot(empty);
        __syncthreads();
        if (lane == 0)
            lds[w] = __popcll(word);
        __syncthreads();
        int r = taken + __popcll(word & ((uint64_t{1} << lane) - 1));
        for (int x = 0; x < w; ++x)
            r += lds[x];
        taken += lds[0] + lds[1] + lds[2] + lds[3];
        if (empty) {
            const int e_new = list[r - first];
            if (e_new >= 0)
                atomicAdd(&a.p.uses_out[e_new], 1);
            out[i] = e_new;
        } else if (i < s.to && in != out) {
            out[i] = e;
        }
    }
}

// ---- fork
struct ForkArgs {
    PoolArgs p;
    const int *parents;
    int *lens_out, *copies, *lacking;
    int *again;  // workspace [batch]: an earlier row has the same parent
};

__global__ __launch_bounds__(256) void k_fork_count(ForkArgs a)
{
    __shared__ int lds[4];
    if (static_cast<int>(blockIdx.x) < a.p.chunks)
        return snapshot(a.p, blockIdx.x, lds);
    const int b = (blockIdx.x - a.p.chunks) * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;  // a wavefront per row
    if (b >= a.p.batch)
        return;
    const int parent = a.parents[b];
    int again = 0, need = 0;
    if (parent >= 0 && parent < a.p.batch) {
        for (int i0 = 0; i0 < b && !again; i0 += 64)
            again = __ballot(i0 + lane < b && a.parents[i0 + lane < b ? i0 + lane : 0] == parent) != 0;
        const int len = cached(a.p, parent), part = len & ((1 << a.p.page_shift) - 1);
        need = again && part && is_page(a.p, a.p.table[static_cast<int64_t>(parent) * a.p.max_pages + (len >> a.p.page_shift)]);
    }
    if (lane == 0) {
        a.again[b] = again;
        a.p.needs[b] = need;
    }
}

__global__ __launch_bounds__(256) void k_fork_rows(ForkArgs a)
{
    __shared__ int lds[8], list[1];
    if (a.p.batch == 0) {
        if (threadIdx.x == 0)
            a.lacking[0] = 0;
        return;
    }
    const int b = blockIdx.y, parent = a.parents[b], again = a.again[b], need = a.p.needs[b];
    Balance all(a.p, b);
    const bool goes_on = parent >= 0 && parent < a.p.batch;
    const int len = goes_on ? cached(a.p, parent) : 0, whole = len >> a.p.page_shift;
    const Span part = part_of(a.p, blockIdx.x);
    const int *from = a.p.table + static_cast<int64_t>(goes_on ? parent : 0) * a.p.max_pages;
    const int64_t row = static_cast<int64_t>(b) * a.p.max_pages;
    int fresh = -1;
    if (blockIdx.x == 0 || (need && whole >= part.from && whole < part.to)) {
        all.sum(a.p, b, lds);
        if (need) {
            free_pages(a.p, all.count, b == 0 ? 0 : all.needs, 1, list, lds);
            fresh = list[0];
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            if (b == 0)
                a.lacking[0] = all.needs > all.free ? all.needs - all.free : 0;
            a.lens_out[b] = len;
            a.copies[2 * static_cast<int64_t>(b)] = fresh >= 0 ? from[whole] : -1;
            a.copies[2 * static_cast<int64_t>(b) + 1] = fresh;
        }
    }
    part_entries(part, from, a.p.table + row, [&](int i, int e, int old) {
        if (!goes_on || (again && i >= whole))
            e = -1;
        if (need && i == whole)
            e = fresh;
        e = is_page(a.p, e) ? e : -1;
        if (e != old) {
            if (e >= 0)
                atomicAdd(&a.p.uses_out[e], 1);
            if (is_page(a.p, old))
                atomicSub(&a.p.uses_out[old], 1);
        }
        a.p.table_out[row + i] = e;
    });
}

// ---- compact
struct CompactArgs {
    PoolArgs p;
    int *copies, *live;
};

__global__ __launch_bounds__(256) void k_snapshot(PoolArgs a)
{
    __shared__ int lds[4];
    snapshot(a, blockIdx.x, lds);
}

// Of n used pages: the free pages below n into the list, in order; the move number of the used ones
// from n on, the highest first; how many there are (the free pages in front of page n).
__global__ __launch_bounds__(256) void k_compact_list(CompactArgs a)
{
    __shared__ int lds[4];
    const int chunk = blockIdx.x, w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int live = a.p.num_pages - sum_of(a.p.counts, a.p.chunks, lds);
    if (a.p.num_pages == 0) {
        if (threadIdx.x == 0)
            a.live[0] = 0;
        return;
    }
    const uint64_t mine = a.p.bits[static_cast<int64_t>(chunk) * kWords + lane];
    const int ranks = words_before(mine, sum_of(a.p.counts, chunk, lds));
    if (chunk == 0 && threadIdx.x == 0) {
        a.live[0] = live;
        if (live == a.p.num_pages)
            a.p.moves[0] = 0;
    }
    for (int i = w; i < kWords; i += 4) {
        const uint64_t word = __shfl(mine, i);
        const int64_t p = static_cast<int64_t>(chunk) * kChunk + 64 * i + lane;
        const int rank = __shfl(ranks, i);
        if (p < a.p.num_pages) {
            const int before = rank + __popcll(word & ((uint64_t{1} << lane) - 1));
            const bool free = word >> lane & 1;
            if (p >= live)
                a.p.map[p] = free ? -1 : live - 1 - (static_cast<int>(p) - before);
            else if (free)
                a.p.list[before] = static_cast<int>(p);
            if (p == live)
                a.p.moves[0] = before;
        }
    }
}

__global__ __launch_bounds__(256) void k_compact_move(CompactArgs a)
{
    __shared__ int lds[4];
    const int live = a.p.num_pages - sum_of(a.p.counts, a.p.chunks, lds);
    if (static_cast<int>(blockIdx.x) < a.p.chunks) {
        const int moves = a.p.moves[0], most = a.p.num_pages / 2;
        for (int x = threadIdx.x; x < kChunk; x += 256) {
            const int64_t p = static_cast<int64_t>(blockIdx.x) * kChunk + x;
            if (p >= moves && p < most)
                a.copies[2 * p] = a.copies[2 * p + 1] = -1;
            if (p < live || p >= a.p.num_pages)
                continue;
            const int r = a.p.map[p];
            if (r < 0)
                continue;
            const int to = a.p.list[r];
            a.p.uses_out[to] = a.p.uses_out[p];
            a.p.uses_out[p] = 0;
            a.copies[2 * static_cast<int64_t>(r)] = static_cast<int>(p);
            a.copies[2 * static_cast<int64_t>(r) + 1] = to;
        }
        return;
    }
    const int64_t all = static_cast<int64_t>(a.p.batch) * a.p.max_pages;
    const int64_t step = static_cast<int64_t>(gridDim.x - a.p.chunks) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x - a.p.chunks) * 256 + threadIdx.x; i < all; i += step) {
        const int e = a.p.table[i];
        int to = is_page(a.p, e) ? e : -1;
        if (to >= live) {
            const int r = a.p.map[e];
            to = r < 0 ? e : a.p.list[r];
        }
        if (to != e || a.p.table_out != a.p.table)
            a.p.table_out[i] = to;
    }
}

// ---- one workgroup
// The same calls where the pool, the table and the streams are small: one launch, since more cost more
// than the work. Free pages and uses are held in LDS. Limits of pages and table entries together: an
// advance of few takes 4.8 us here and 8.4 as two launches, of 16,000 9.0 and 9.4, of 32,000 14.2 and
// 9.6; a compaction, three launches else, of 32,000 11.6 and 15.6, of 80,000 18.8 and 15.0.
constexpr int kSmallPages = 16384, kSmallRows = 1024, kSmallThreads = 1024, kSmallWaves = kSmallThreads / 64;
constexpr int64_t kSmallTake = 16384, kSmallCompact = 49152;

struct Small {
    int list[kSmallPages];  // free pages in order; compact: where a page goes, from page n on
    int uses[kSmallPages];
    uint64_t bits[kSmallPages / 64];
    int before[kSmallPages / 64];  // free pages in front of a word
    int rows[3][kSmallRows];
    int sums[kSmallWaves];
};

// Exclusive sums of v over the workgroup's threads; the whole sum in `all`.
__device__ __forceinline__ int sums_before(int v, int *lds, int *all)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int n = v;
#pragma unroll
    for (int y = 1; y < 64; y *= 2) {
        const int o = __shfl_up(n, y);
        n += lane >= y ? o : 0;
    }
    __syncthreads();  // lds may still be read from an earlier sum
    if (lane == 63)
        lds[w] = n;
    __syncthreads();
    int front = 0, whole = 0;
#pragma unroll
    for (int x = 0; x < kSmallWaves; ++x) {
        front += x < w ? lds[x] : 0;
        whole += lds[x];
    }
    *all = whole;
    return front + n - v;
}

// Uses and free bits into LDS, and the free pages in front of every word. Returns how many there are.
__device__ __forceinline__ int small_snapshot(const PoolArgs &a, Small &m)
{
    const int lane = threadIdx.x & 63, words = (a.num_pages + 63) / 64;
    int u[kSmallPages / kSmallThreads];
#pragma unroll
    for (int k = 0; k < kSmallPages / kSmallThreads; ++k) {
        const int p = threadIdx.x + k * kSmallThreads;
        u[k] = 1;
        if (k * kSmallThreads < a.num_pages)
            u[k] = a.uses[p < a.num_pages ? p : a.num_pages - 1];
    }
#pragma unroll
    for (int k = 0; k < kSmallPages / kSmallThreads; ++k) {
        const int p = threadIdx.x + k * kSmallThreads;
        if (k * kSmallThreads >= a.num_pages)
            break;
        const uint64_t word = __ballot(p < a.num_pages && u[k] <= 0);
        if (p < words * 64)
            m.uses[p] = u[k] > 0 ? u[k] : 0;
        if (lane == 0 && p < words * 64)
            m.bits[p / 64] = word;
    }
    __syncthreads();
    const int x = threadIdx.x;
    int free;
    const int n = sums_before(x < words ? __popcll(m.bits[x]) : 0, m.sums, &free);
    if (x < words)
        m.before[x] = n;
    __syncthreads();
    return free;
}

__device__ __forceinline__ int free_before(const Small &m, int p)
{
    return m.before[p / 64] + __popcll(m.bits[p / 64] & ((uint64_t{1} << (p & 63)) - 1));
}

// the first `most` free pages, in order
__device__ __forceinline__ void small_list(const PoolArgs &a, Small &m, int most)
{
    for (int p = threadIdx.x; p < a.num_pages; p += kSmallThreads) {
        if (!(m.bits[p / 64] >> (p & 63) & 1))
            continue;
        const int r = free_before(m, p);
        if (r < most)
            m.list[r] = p;
    }
    __syncthreads();
}

__device__ __forceinline__ void small_uses_out(const PoolArgs &a, const Small &m)
{
    for (int p = threadIdx.x; p < a.num_pages; p += kSmallThreads)
        a.uses_out[p] = m.uses[p];
}

// f(y, entry y of table[0 .. n)), or of both tables, for the entries of a thread; eight are loaded
// before the first is used.
template <typename F>
__device__ __forceinline__ void small_entries(const int *table, int n, F f)
{
    constexpr int U = 8;
    for (int y0 = threadIdx.x; y0 < n; y0 += U * kSmallThreads) {
        int e[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int y = y0 + k * kSmallThreads;
            e[k] = table[y < n ? y : n - 1];
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (y0 + k * kSmallThreads < n)
                f(y0 + k * kSmallThreads, e[k]);
    }
}

__global__ __launch_bounds__(kSmallThreads) void k_advance_small(AdvanceArgs a, Divisor by_row)
{
    __shared__ Small m;
    const int x = threadIdx.x, per = a.p.max_pages;
    // a stream per thread: what its new tokens start, and how many of those entries are empty
    Span s{};
    int empty = 0;
    if (x < a.p.batch) {
        s = new_entries(a, x);
        for (int i = s.from; i < s.to; ++i)
            empty += !is_page(a.p, a.p.table[x * per + i]);
        m.rows[0][x] = s.from, m.rows[1][x] = s.to, m.rows[2][x] = s.len;
    }
    const int free = small_snapshot(a.p, m);
    int need;
    int place = sums_before(empty, m.sums, &need);
    small_list(a.p, m, need);
    for (int i = s.from; i < s.to; ++i) {  // the stream's own thread; others have an empty span
        const int e = a.p.table[x * per + i];
        int to = e;
        if (!is_page(a.p, e)) {
            to = place < free ? m.list[place] : -1;
            ++place;
            if (to >= 0)
                atomicAdd(&m.uses[to], 1);
        }
        if (to != e || a.p.table_out != a.p.table)
            a.p.table_out[x * per + i] = to;
    }
    small_entries(a.p.table, a.p.batch * per, [&](int y, int e) {
        const int b = by_row(y), i = y - b * per;
        const Span r = {m.rows[0][b], m.rows[1][b], m.rows[2][b]};
        if (i >= r.from && i < r.to)
            return;
        const bool kept = stays(a, r, i, e);
        if (!kept && is_page(a.p, e))
            atomicSub(&m.uses[e], 1);
        if (a.p.table != a.p.table_out || !kept)
            a.p.table_out[y] = kept ? e : -1;
    });
    __syncthreads();
    small_uses_out(a.p, m);
    if (x == 0)
        a.lacking[0] = need > free ? need - free : 0;
}

__global__ __launch_bounds__(kSmallThreads) void k_fork_small(ForkArgs a, Divisor by_row)
{
    __shared__ Small m;
    const int x = threadIdx.x, per = a.p.max_pages;
    int *const first = m.rows[2];  // the first row with this parent
    const int parent = x < a.p.batch ? a.parents[x] : -1;
    const bool goes_on = parent >= 0 && parent < a.p.batch;
    first[x] = INT_MAX;
    __syncthreads();
    if (goes_on)
        atomicMin(&first[parent], x);
    const int free = small_snapshot(a.p, m);
    const int len = goes_on ? cached(a.p, parent) : 0, whole = len >> a.p.page_shift;
    const bool again = goes_on && first[parent] != x;
    int old = -1;
    if (again && (len & ((1 << a.p.page_shift) - 1)))
        old = a.p.table[parent * per + whole];
    old = is_page(a.p, old) ? old : -1;
    int need;
    const int place = sums_before(old >= 0, m.sums, &need);
    small_list(a.p, m, need);
    const int fresh = old >= 0 && place < free ? m.list[place] : -1;
    if (x < a.p.batch) {
        a.lens_out[x] = len;
        a.copies[2 * x] = fresh >= 0 ? old : -1;
        a.copies[2 * x + 1] = fresh;
        m.rows[0][x] = again ? whole : per;  // entries from here on are not the parent's
        m.rows[1][x] = goes_on ? parent : -1;
        m.rows[2][x] = fresh;  // every thread has read `first` before the list's last barrier
    }
    __syncthreads();
    // the parents' entries, and what they replace; eight of a thread loaded before the first is used
    constexpr int U = 8;
    const int all = a.p.batch * per;
    for (int y0 = x; y0 < all; y0 += U * kSmallThreads) {
        int now[U], old[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int y = min(y0 + k * kSmallThreads, all - 1), b = by_row(y), p = m.rows[1][b];
            old[k] = a.p.table[y];
            now[k] = a.p.table[p < 0 ? y : p * per + y - b * per];
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int y = y0 + k * kSmallThreads;
            if (y >= all)
                break;
            const int b = by_row(y), i = y - b * per, from = m.rows[0][b], was = old[k];
            int e = m.rows[1][b] >= 0 && i < from ? now[k] : -1;
            if (i == from)
                e = m.rows[2][b];
            e = is_page(a.p, e) ? e : -1;
            if (e != was) {
                if (e >= 0)
                    atomicAdd(&m.uses[e], 1);
                if (is_page(a.p, was))
                    atomicSub(&m.uses[was], 1);
            }
            a.p.table_out[y] = e;
        }
    }
    __syncthreads();
    small_uses_out(a.p, m);
    if (x == 0)
        a.lacking[0] = need > free ? need - free : 0;
}

__global__ __launch_bounds__(kSmallThreads) void k_compact_small(CompactArgs a)
{
    __shared__ Small m;
    const int x = threadIdx.x, P = a.p.num_pages;
    const int live = P - small_snapshot(a.p, m), moves = live < P ? free_before(m, live) : 0;
    small_list(a.p, m, moves);
    // where the pages from `live` on go: behind the list, which ends at moves <= live
    for (int p = live + x; p < P; p += kSmallThreads) {
        if (m.bits[p / 64] >> (p & 63) & 1)
            m.list[p] = p;
        else {
            const int r = live - 1 - (p - free_before(m, p)), to = m.list[r];
            m.list[p] = to;
            m.uses[to] = m.uses[p];
            m.uses[p] = 0;
            a.copies[2 * r] = p, a.copies[2 * r + 1] = to;
        }
    }
    for (int r = moves + x; r < P / 2; r += kSmallThreads)
        a.copies[2 * r] = a.copies[2 * r + 1] = -1;
    __syncthreads();
    small_entries(a.p.table, a.p.batch * a.p.max_pages, [&](int y, int e) {
        int to = is_page(a.p, e) ? e : -1;
        to = to >= live ? m.list[to] : to;
        if (to != e || a.p.table_out != a.p.table)
            a.p.table_out[y] = to;
    });
    small_uses_out(a.p, m);
    if (x == 0)
        a.live[0] = live;
}

// ---- copies
// A workgroup takes 16 KB of a page of one pool: entries along x, pools and parts along y. Threads
// past the page's end read its last piece again, so that no load is conditional: a conditional one
// per piece made the compiler keep the pieces in LDS and wait for each (800 pages of 32 KB: 25.7 us,
// and 16 us for a list that names none; 16.5 and 2 so). Stores do not stay in the L2s: what a pool of
// pages that were last used long ago needs, a compaction of 187 MB moved, 50 us, 41 so; loads that do
// not stay either 46, they alone 42. 800 pages of 64 KB: 31.4 us, 6.7 TB/s both ways.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kPieces = 4;  // 16-byte pieces of a thread

__global__ __launch_bounds__(256) void k_pages_copy(char *k, char *v, const int *copies, int n, int step, int num_pages,
                                                    int64_t page_bytes)
{
    char *pool = blockIdx.y & 1 ? v : k;
    const int64_t at = (static_cast<int64_t>(blockIdx.y >> 1) * kPieces * 256 + threadIdx.x) * 16;
    for (int64_t i = blockIdx.x; i < n; i += step) {
        const int from = copies[2 * i], to = copies[2 * i + 1];
        if (from < 0 || to < 0 || from >= num_pages || to >= num_pages || from == to)
            continue;
        const char *src = pool + from * page_bytes;
        char *dst = pool + to * page_bytes;
        auto read = [&](int x) {
            const int64_t o = at + x * 4096;
            return *reinterpret_cast<const u32x4 *>(src + (o < page_bytes ? o : page_bytes - 16));
        };
        const u32x4 d0 = read(0), d1 = read(1), d2 = read(2), d3 = read(3);
        auto write = [&](int x, u32x4 d) {
            if (at + x * 4096 < page_bytes)
                __builtin_nontemporal_store(d, reinterpret_cast<u32x4 *>(dst + at + x * 4096));
        };
        write(0, d0), write(1, d1), write(2, d2), write(3, d3);
    }
}

// ---- host
bdssm_status check_pages_dims(const bdssm_pages_dims *d)
{
    if (!d)
        return BDSSM_ERR_NULL;
    if (d->batch < 0 || d->num_pages < 0 || d->max_pages < 0)
        return BDSSM_ERR_SHAPE;
    const int p = d->page_size;
    if ((p != 16 && p != 32 && p != 64 && p != 128 && p != 256) || d->batch > 65535 ||
        static_cast<int64_t>(d->max_pages) * p > kMaxPosition)
        return BDSSM_ERR_UNSUPPORTED;
    return BDSSM_OK;
}

// Whether one workgroup takes a call: what it holds in LDS, and as long as pages and table entries
// together are no more than `most`.
bool small(const bdssm_pages_dims *d, int64_t most)
{
    return d->num_pages <= kSmallPages && d->batch <= kSmallRows &&
           d->num_pages + static_cast<int64_t>(d->batch) * d->max_pages <= most;
}

int64_t chunks_of(const bdssm_pages_dims *d) { return (static_cast<int64_t>(d->num_pages) + kChunk - 1) / kChunk; }

// Bytes of the workspace, and with `a` and `again` the places in it.
size_t workspace_of(const bdssm_pages_dims *d, char *ws, PoolArgs *a, int **again)
{
    int64_t used = 0;
    auto take = [&](int64_t bytes) {
        char *at = ws ? ws + used : nullptr;
        used += (bytes + 15) / 16 * 16;
        return at;
    };
    PoolArgs none;
    int *skip;
    a = a ? a : &none, again = again ? again : &skip;
    a->bits = reinterpret_cast<uint64_t *>(take(chunks_of(d) * kWords * 8));
    a->counts = reinterpret_cast<int *>(take(chunks_of(d) * 4));
    a->needs = reinterpret_cast<int *>(take(d->batch * 4ll));
    *again = reinterpret_cast<int *>(take(d->batch * 4ll));
    a->list = reinterpret_cast<int *>(take(d->num_pages * 4ll));
    a->map = reinterpret_cast<int *>(take(d->num_pages * 4ll));
    a->moves = reinterpret_cast<int *>(take(4));
    return static_cast<size_t>(used);
}

// What the three calls check alike: pointers, alignment, overlaps (of the inputs in `in`, the outputs
// in `out`; the first output is table_out, the second uses_out, which may be in place), workspace.
bdssm_status prepare_pages(const bdssm_pages_dims *d, const bdssm_pages *g, const int32_t *extra_in, int64_t extra_count,
                           bool need_extra, int32_t *const (&out)[5], const int64_t (&count)[5], bool table_in_place,
                           void *ws, size_t ws_bytes, PoolArgs *a, int **again)
{
    const bdssm_status rc = check_pages_dims(d);
    if (rc != BDSSM_OK)
        return rc;
    if (!g)
        return BDSSM_ERR_NULL;
    const int64_t entries = static_cast<int64_t>(d->batch) * d->max_pages;
    const Range in[4] = {rng(g->table, entries * 4), rng(g->uses, d->num_pages * 4ll), rng(g->lens, d->batch * 4ll),
                         rng(extra_in, extra_count * 4)};
    if ((!g->table && entries > 0) || (!g->uses && d->num_pages > 0) || (!g->lens && d->batch > 0) ||
        (need_extra && !extra_in && extra_count > 0))
        return BDSSM_ERR_NULL;
    for (int i = 0; i < 5; ++i)
        if (!out[i] && count[i] > 0)
            return BDSSM_ERR_NULL;
    if (!aligned4(g->table) || !aligned4(g->uses) || !aligned4(g->lens) || !aligned4(extra_in) || !aligned(ws))
        return BDSSM_ERR_ALIGN;
    for (int i = 0; i < 5; ++i)
        if (!aligned4(out[i]))
            return BDSSM_ERR_ALIGN;
    for (int i = 0; i < 5; ++i) {
        const Range w = rng(out[i], count[i] * 4);
        for (int j = 0; j < 4; ++j) {
            const bool in_place = i == j && (i == 1 || (i == 0 && table_in_place)) && w.lo == in[j].lo;
            if (!in_place && overlap(w, in[j]))
                return BDSSM_ERR_ALIAS;
        }
        for (int j = 0; j < i; ++j)
            if (overlap(w, rng(out[j], count[j] * 4)))
                return BDSSM_ERR_ALIAS;
    }
    *a = PoolArgs{};
    const size_t need = workspace_of(d, static_cast<char *>(ws), a, again);
    if (!ws || ws_bytes < need)
        return BDSSM_ERR_WORKSPACE;
    const Range rw = rng(ws, static_cast<int64_t>(need));
    for (const Range &x : in)
        if (overlap(rw, x))
            return BDSSM_ERR_ALIAS;
    for (int i = 0; i < 5; ++i)
        if (overlap(rw, rng(out[i], count[i] * 4)))
            return BDSSM_ERR_ALIAS;
    a->table = g->table, a->lens = g->lens, a->uses = g->uses;
    a->table_out = out[0], a->uses_out = out[1];
    a->batch = d->batch, a->page_shift = __builtin_ctz(d->page_size);
    a->num_pages = d->num_pages, a->max_pages = d->max_pages;
    a->chunks = static_cast<int>(chunks_of(d));
    // parts of a row: a thousand entries or more each, as many as fill the GPU
    a->row_parts = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>((d->max_pages + 1023) / 1024, 1024 / std::max(1, d->batch))));
    return BDSSM_OK;
}

}  // namespace
}  // namespace bdssm

using namespace bdssm;

extern "C" size_t bdssm_pages_workspace(const bdssm_pages_dims *dims)
{
    return check_pages_dims(dims) == BDSSM_OK ? workspace_of(dims, nullptr, nullptr, nullptr) : SIZE_MAX;
}

extern "C" bdssm_status bdssm_pages_advance(const bdssm_pages_dims *dims, const bdssm_pages *pages, const int32_t *starts,
                                            int32_t block_len, int32_t window, int32_t sinks, int32_t *table_out,
                                            int32_t *uses_out, int32_t *lacking, void *workspace, size_t workspace_bytes,
                                            void *stream)
{
    AdvanceArgs a{};
    int *again;
    const int64_t batch = dims ? dims->batch : 0;
    int32_t *const out[5] = {table_out, uses_out, lacking, nullptr, nullptr};
    const int64_t count[5] = {dims ? batch * dims->max_pages : 0, dims ? dims->num_pages : 0, 1, 0, 0};
    const bdssm_status rc = prepare_pages(dims, pages, starts, batch + 1, false, out, count, true, workspace,
                                          workspace_bytes, &a.p, &again);
    if (rc != BDSSM_OK)
        return rc;
    if (block_len < 0 || window < 0 || sinks < 0)
        return BDSSM_ERR_SHAPE;
    // entries that new tokens start, of all streams, are counted in 32 bits
    if (batch * std::min(dims->max_pages, block_len / dims->page_size + 1) > INT_MAX)
        return BDSSM_ERR_UNSUPPORTED;
    a.starts = starts, a.block_len = block_len, a.window = window, a.sinks = sinks, a.lacking = lacking;
    hipStream_t st = static_cast<hipStream_t>(stream);
    // a stream's new entries are one thread's there
    if (small(dims, kSmallTake) && block_len / dims->page_size <= 64) {
        k_advance_small<<<1, kSmallThreads, 0, st>>>(a, Divisor(std::max(1, dims->max_pages)));
        return launched(hipGetLastError());
    }
    if (a.p.chunks + dims->batch > 0)
        k_advance_count<<<a.p.chunks + dims->batch, 256, 0, st>>>(a);
    k_advance_rows<<<dim3(a.p.row_parts + (a.p.row_parts > 1), std::max(1, dims->batch)), 256, 0, st>>>(a);
    return launched(hipGetLastError());
}

extern "C" bdssm_status bdssm_pages_fork(const bdssm_pages_dims *dims, const bdssm_pages *pages, const int32_t *parents,
                                         int32_t *table_out, int32_t *lens_out, int32_t *uses_out, int32_t *copies,
                                         int32_t *lacking, void *workspace, size_t workspace_bytes, void *stream)
{
    ForkArgs a{};
    const int64_t batch = dims ? dims->batch : 0;
    int32_t *const out[5] = {table_out, uses_out, lens_out, copies, lacking};
    const int64_t count[5] = {dims ? batch * dims->max_pages : 0, dims ? dims->num_pages : 0, batch, 2 * batch, 1};
    const bdssm_status rc = prepare_pages(dims, pages, parents, batch, true, out, count, false, workspace, workspace_bytes,
                                          &a.p, &a.again);
    if (rc != BDSSM_OK)
        return rc;
    a.parents = parents, a.lens_out = lens_out, a.copies = copies, a.lacking = lacking;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (small(dims, kSmallTake)) {
        k_fork_small<<<1, kSmallThreads, 0, st>>>(a, Divisor(std::max(1, dims->max_pages)));
        return launched(hipGetLastError());
    }
    const int rows = (dims->batch + 3) / 4;
    if (a.p.chunks + rows > 0)
        k_fork_count<<<a.p.chunks + rows, 256, 0, st>>>(a);
    k_fork_rows<<<dim3(a.p.row_parts, std::max(1, dims->batch)), 256, 0, st>>>(a);
    return launched(hipGetLastError());
}

extern "C" bdssm_status bdssm_pages_compact(const bdssm_pages_dims *dims, const bdssm_pages *pages, int32_t *table_out,
                                            int32_t *uses_out, int32_t *copies, int32_t *live, void *workspace,
                                            size_t workspace_bytes, void *stream)
{
    CompactArgs a{};
    int *again;
    const int64_t entries = dims ? static_cast<int64_t>(dims->batch) * dims->max_pages : 0;
    int32_t *const out[5] = {table_out, uses_out, copies, live, nullptr};
    const int64_t count[5] = {entries, dims ? dims->num_pages : 0, dims ? dims->num_pages / 2 * 2ll : 0, 1, 0};
    const bdssm_status rc = prepare_pages(dims, pages, nullptr, 0, false, out, count, true, workspace, workspace_bytes, &a.p,
                                          &again);
    if (rc != BDSSM_OK)
        return rc;
    a.copies = copies, a.live = live;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (small(dims, kSmallCompact)) {
        k_compact_small<<<1, kSmallThreads, 0, st>>>(a);
        return launched(hipGetLastError());
    }
    if (a.p.chunks > 0)
        k_snapshot<<<a.p.chunks, 256, 0, st>>>(a.p);
    k_compact_list<<<std::max(1, a.p.chunks), 256, 0, st>>>(a);
    const int rows = static_cast<int>(std::min<int64_t>(1024, (entries + 1023) / 1024));
    if (a.p.chunks + rows > 0)
        k_compact_move<<<a.p.chunks + rows, 256, 0, st>>>(a);
    return launched(hipGetLastError());
}

extern "C" bdssm_status bdssm_pages_copy(const bdssm_attn_dims *dims, const bdssm_kv_cache *cache, const int32_t *copies,
                                         int32_t n, void *stream)
{
    const bdssm_status rc = check_attn_dims(dims);
    if (rc != BDSSM_OK)
        return rc;
    if (!cache)
        return BDSSM_ERR_NULL;
    if (cache->num_pages < 0 || n < 0)
        return BDSSM_ERR_SHAPE;
    if ((n > 0 && !copies) || (cache->num_pages > 0 && (!cache->k || !cache->v)))
        return BDSSM_ERR_NULL;
    if (!aligned4(copies) || !aligned(cache->k) || !aligned(cache->v))
        return BDSSM_ERR_ALIGN;
    const int64_t page_bytes = static_cast<int64_t>(dims->kv_heads) * dims->page_size * dims->headdim * elt(dims->dtype);
    const Range k = rng(cache->k, cache->num_pages * page_bytes), v = rng(cache->v, cache->num_pages * page_bytes);
    const Range rc_ = rng(copies, n * 8ll);
    if (overlap(k, v) || overlap(rc_, k) || overlap(rc_, v))
        return BDSSM_ERR_ALIAS;
    if (n == 0 || cache->num_pages == 0)
        return BDSSM_OK;
    const int64_t parts = 2 * ((page_bytes + kPieces * 4096 - 1) / (kPieces * 4096));  // 8,192 for the largest page
    const int64_t lists = std::min<int64_t>(n, std::max<int64_t>(1, 16384 / parts));
    k_pages_copy<<<dim3(static_cast<unsigned>(lists), static_cast<unsigned>(parts)), 256, 0, static_cast<hipStream_t>(stream)>>>(
        static_cast<char *>(cache->k), static_cast<char *>(cache->v), copies, n, static_cast<int>(lists), cache->num_pages, page_bytes);
    return launched(hipGetLastError());
}
