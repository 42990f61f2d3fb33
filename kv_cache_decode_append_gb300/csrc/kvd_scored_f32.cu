// Instantiates the fp32 attention kernels with modified scores, the separate merge pass.
#include "kvd_attention.cuh"

namespace kvd {
bool attn_variant_scored_f32(int D, int RB, bool paged, AttnVariant *v)
{
    return pick_scored_variant<float, false>(D, RB, paged, v);
}
}  // namespace kvd
