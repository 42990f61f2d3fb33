// Instantiates the f16 shared-prefix kernels (tcgen05) and their join.
#include "kvd_pair_tc5.cuh"

namespace kvd {
bool prefix_variant_f16(int D, bool paged, PrefixVariant *v) { return pick_pair_prefix<__half>(D, paged, v); }
}  // namespace kvd
