// Instantiates the bf16 attention kernels with modified scores, split heads merged inside the kernel:
// CUDA cores (RB 1 .. 8), mma.sync (RB 16), tcgen05 (RB 128).
#include "kvd_attention.cuh"
#include "kvd_attention_mma.cuh"
#include "kvd_attention_tc5.cuh"

namespace kvd {
bool attn_variant_scored_bf16_tk(int D, int RB, bool paged, AttnVariant *v)
{
    if (RB == 128) return pick_scored_tc5_variant<__nv_bfloat16, true>(D, paged, v);
    if (RB == 16) return pick_scored_mma_variant<__nv_bfloat16, true>(D, paged, v);
    return pick_scored_variant<__nv_bfloat16, true>(D, RB, paged, v);
}
}  // namespace kvd
