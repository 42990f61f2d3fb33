// Instantiates the bf16 tcgen05 attention kernels with modified scores (RB 128),
// split heads merged inside the kernel.
#include "kvd_attention_tc5.cuh"

namespace kvd {
bool attn_variant_scored_bf16_tk(int D, int RB, bool paged, AttnVariant *v)
{
    return RB == 128 && pick_scored_tc5_variant<__nv_bfloat16, true>(D, paged, v);
}
}  // namespace kvd
