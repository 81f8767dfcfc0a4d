// Attention of a chunk over a paged cache with ranges of each row and a bias by distance
// (bdssm_attn_step_ex): the kernels of attn_kernel.h, a unit to each of their modes; and the order of row
// tiles, for every mode that has ranges.
#include "attn_kernel.h"

namespace bdssm {
namespace {

// The row tiles of a stream whose rows have ranges, the longest first: what a tile has to walk is in
// device memory, and workgroups that take more than one round end together only so (documents of 350
// to 1,050 tokens in a prompt: without it some CUs had twice the average). A tile counts as the keys
// from its first row's lower to its last row's upper bound; 1,024 classes of them are sorted by
// counting, in no order inside a class (row tiles do not depend on one another).
__global__ __launch_bounds__(1024) void k_attn_order(AttnArgs a, int nrt, int rows, int tk, int shift, int *order)
{
    __shared__ int at[1024], sums[16];
    const int b = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const AttnStream s = attn_stream(a, b);
    const int end = s.len + (a.k ? s.n : 0), prefix = prefix_of(a, b, end), G = static_cast<int>(a.by_group.d);
    const int64_t all = static_cast<int64_t>(s.n) * G;
    auto kind = [&](int rt) {  // 0: the longest
        const int64_t r0 = static_cast<int64_t>(rt) * rows, r1 = r0 + rows < all ? r0 + rows : all;
        int keys = 0;
        if (r0 < r1) {
            const Sight x = sight_of<true>(a, s, end, prefix, a.by_group(static_cast<int>(r0)));
            const Sight y = sight_of<true>(a, s, end, prefix, a.by_group(static_cast<int>(r1 - 1)));
            const int lo = x.lo < y.lo ? x.lo : y.lo, hi = x.hi > y.hi ? x.hi : y.hi;
            keys = lo < hi ? hi - lo : 0;
        }
        const int tiles = (keys / tk + (keys > 0)) >> shift;
        return 1023 - (tiles < 1023 ? tiles : 1023);
    };
    at[threadIdx.x] = 0;
    __syncthreads();
    for (int rt = threadIdx.x; rt < nrt; rt += 1024)
        atomicAdd(&at[kind(rt)], 1);
    __syncthreads();
    const int mine = at[threadIdx.x];
    int n = mine;
#pragma unroll
    for (int y = 1; y < 64; y *= 2) {
        const int o = __shfl_up(n, y);
        n += lane >= y ? o : 0;
    }
    if (lane == 63)
        sums[w] = n;
    __syncthreads();
    for (int x = 0; x < w; ++x)
        n += sums[x];
    at[threadIdx.x] = n - mine;
    __syncthreads();
    for (int rt = threadIdx.x; rt < nrt; rt += 1024)
        order[static_cast<int64_t>(b) * nrt + atomicAdd(&at[kind(rt)], 1)] = rt;
}

}  // namespace

void launch_attn_order(const AttnArgs &a, int nrt, int rows, int tk, int shift, int *order, hipStream_t st)
{
    k_attn_order<<<a.batch, 1024, 0, st>>>(a, nrt, rows, tk, shift, order);
}

hipError_t launch_attn_ranged(const AttnArgs &a, int D, bool bf16, const AttnPlan &p, void *ws, hipStream_t st)
{
    return by_type(a, D, bf16, Launch<kRanged>{a, p, ws, st});
}

}  // namespace bdssm
