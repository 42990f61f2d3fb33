// Instantiates the bf16 shared-prefix kernels (tcgen05) and their join.
#include "kvd_pair_tc5.cuh"

namespace kvd {
bool prefix_variant_bf16(int D, bool paged, PrefixVariant *v) { return pick_pair_prefix<__nv_bfloat16>(D, paged, v); }
}  // namespace kvd
