// Attention of a chunk over a paged cache with shaped scores or ranges of each token's own
// (bdssm_attn_step_ex): the kernels of attn_kernel.h, built apart from those for plain scores.
#include "attn_kernel.h"

namespace bdssm {

hipError_t launch_attn_scored(const AttnArgs &a, int D, bool bf16, const AttnPlan &p, void *ws, hipStream_t st)
{
    return by_type(D, bf16, static_cast<int64_t>(a.block_len) * (a.H / a.KV), Launch<true>{a, p, ws, st});
}

}  // namespace bdssm
