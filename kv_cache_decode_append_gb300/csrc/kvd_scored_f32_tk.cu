// Instantiates the fp32 attention kernels with modified scores, split heads merged inside the kernel.
#include "kvd_attention.cuh"

namespace kvd {
bool attn_variant_scored_f32_tk(int D, int RB, bool paged, AttnVariant *v)
{
    return pick_scored_variant<float, true>(D, RB, paged, v);
}
}  // namespace kvd
