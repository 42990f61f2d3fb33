// Instantiates the f16 tcgen05 attention kernels with modified scores (RB 128),
// the separate merge pass.
#include "kvd_attention_tc5.cuh"

namespace kvd {
bool attn_variant_scored_f16(int D, int RB, bool paged, AttnVariant *v)
{
    return RB == 128 && pick_scored_tc5_variant<__half, false>(D, paged, v);
}
}  // namespace kvd
