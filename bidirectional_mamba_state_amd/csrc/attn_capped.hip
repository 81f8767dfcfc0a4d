// Attention of a chunk over a paged cache with capped scores, and ranges and a bias where they are given
// (bdssm_attn_step_ex): the kernels of attn_kernel.h, a unit to each of their modes.
#include "attn_kernel.h"

namespace bdssm {

hipError_t launch_attn_capped(const AttnArgs &a, int D, bool bf16, const AttnPlan &p, void *ws, hipStream_t st)
{
    return by_type(a, D, bf16, Launch<kCapped>{a, p, ws, st});
}

}  // namespace bdssm
