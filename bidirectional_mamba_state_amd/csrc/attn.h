// Attention over a paged cache: kernel arguments and the device-side view of a stream shared by
// the attention kernels and the append (include/bdssm.h states the layouts and the mask).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace bdssm {

// Division of n in [0, 2^31) by a number the host knows: with k = ceil(log2 d) and
// mul = floor(2^(31+k) / d) + 1, floor(n mul / 2^(31+k)) = floor(n / d), since mul d exceeds
// 2^(31+k) by at most d <= 2^k, which n < 2^31 cannot make a whole 2^(31+k). A kernel's start
// has some twenty divisions, and each would take thirty instructions.
struct Divisor {
    uint32_t d = 1, mul = 0, shift = 0;  // mul 0: d is 1
    Divisor() = default;
    explicit Divisor(int64_t by) : d(static_cast<uint32_t>(by))
    {
        if (d <= 1)
            return;
        const int k = 32 - __builtin_clz(d - 1);
        mul = static_cast<uint32_t>((uint64_t{1} << (31 + k)) / d + 1);
        shift = k - 1;
    }
    __host__ __device__ __forceinline__ int operator()(int n) const
    {
        const uint32_t u = static_cast<uint32_t>(n);
        return static_cast<int>(mul ? static_cast<uint32_t>(static_cast<uint64_t>(u) * mul >> 32) >> shift : u);
    }
    __host__ __device__ __forceinline__ int rest(int n) const { return n - (*this)(n) * static_cast<int>(d); }
};

struct AttnArgs {
    const void *q, *k, *v;  // chunk rows; k, v NULL: no keys of its own
    int64_t q_stride, k_stride, v_stride;
    int64_t tokens;
    const int *starts;  // NULL: uniform
    int block_len;
    void *kp, *vp;  // pools of pages
    const int *table, *lens;
    int num_pages, max_pages, max_len;
    int batch, H, KV, page_shift;
    float scale;
    int block, window, sinks;
    Divisor by_block, by_group;  // block (1 where it is 0), H / KV
    void *out;
};

// One stream's chunk rows and cached tokens. Every count read from device memory is brought
// into the bounds the host knows, so that no index built from it leaves a buffer.
struct AttnStream {
    int64_t row0;  // first chunk row
    int n;         // chunk tokens
    int len;       // cached tokens
};

__device__ __forceinline__ AttnStream attn_stream(const AttnArgs &a, int b)
{
    AttnStream s;
    const int len = a.lens[b];
    s.len = len < 0 ? 0 : len > a.max_len ? a.max_len : len;
    if (!a.starts) {
        s.row0 = static_cast<int64_t>(b) * a.block_len;
        s.n = a.block_len;
        return s;
    }
    int64_t r0 = a.starts[b], r1 = a.starts[b + 1];
    r0 = r0 < 0 ? 0 : r0 > a.tokens ? a.tokens : r0;
    r1 = r1 < r0 ? r0 : r1 > a.tokens ? a.tokens : r1;
    s.row0 = r0;
    s.n = static_cast<int>(r1 - r0 < a.block_len ? r1 - r0 : a.block_len);
    return s;
}

constexpr int64_t kMaxGroups = (int64_t{1} << 32) / 512 - 1;  // a grid's threads have to fit 32 bits

// Launch plan of a step. A unit is one (stream, KV head, range of its keys); its row tiles read
// the same keys, so they go to one XCD (its L2 then fetches them once), side by side in time.
// Few units with many row tiles are cut into `sub` parts of every sub-th tile, so that all eight
// XCDs have work. Workgroup id: XCD id % 8, and inside an XCD row tiles run fastest (rt_fast) or
// slowest.
struct AttnPlan {
    int nrt, nsplit;                   // row tiles per (stream, KV head); ranges of its keys
    int sub, nrt_sub, units, per_xcd;  // parts per unit, row tiles per part, parts, parts per XCD
    int rt_fast;
    Divisor by_inner, by_units, by_kv, by_split;  // nrt_sub or per_xcd, units / sub, KV, nsplit
    int64_t groups;                    // workgroups; more than kMaxGroups cannot be launched
    size_t ml_bytes, ws_bytes;         // workspace: maxima and sums first, then rows (0 unless split)
};

AttnPlan attn_plan(const AttnArgs &a, int D, bool bf16);
// The most that the plan of any length up to a.max_len needs. The plan itself does not grow with
// the length: a longer cache may fit whole rounds of workgroups with fewer ranges. SIZE_MAX: more
// rows than a launch has threads for.
size_t attn_workspace(const AttnArgs &a, int D, bool bf16);
hipError_t launch_attn(const AttnArgs &a, int D, bool bf16, const AttnPlan &p, void *ws, hipStream_t st);

}  // namespace bdssm
