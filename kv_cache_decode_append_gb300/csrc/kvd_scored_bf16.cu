// Instantiates the bf16 tcgen05 kernels with modified scores and their join.
#include "kvd_pair_tc5.cuh"

namespace kvd {
bool pair_variant_bf16(int D, bool paged, PairVariant *v) { return pick_pair_scored<__nv_bfloat16>(D, paged, v); }
}  // namespace kvd
