// Attention of a chunk over a paged cache with ranges of each row and a bias by distance
// (bdssm_attn_step_ex): the kernels of attn_kernel.h, a unit to each of their modes.
#include "attn_kernel.h"

namespace bdssm {

hipError_t launch_attn_ranged(const AttnArgs &a, int D, bool bf16, const AttnPlan &p, void *ws, hipStream_t st)
{
    return by_type(a, D, bf16, Launch<kRanged>{a, p, ws, st});
}

}  // namespace bdssm
