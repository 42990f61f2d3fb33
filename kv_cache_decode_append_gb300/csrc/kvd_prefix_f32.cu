// Instantiates the fp32 shared-prefix kernels and their join.
#include "kvd_prefix_simt.cuh"

namespace kvd {
bool prefix_variant_f32(int D, bool paged, PrefixVariant *v)
{
    if (D == 64) make_prefix_simt<64>(paged, v);
    else if (D == 128) make_prefix_simt<128>(paged, v);
    else return false;
    return true;
}
}  // namespace kvd
