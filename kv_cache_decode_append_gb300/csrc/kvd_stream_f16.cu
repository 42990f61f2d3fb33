// Instantiates the f16 streaming attention kernels with modified scores.
#include "kvd_attention_stream.cuh"

namespace kvd {
const void *stream_kernel_f16(int D, int rows, bool paged) { return pick_stream_kernel<__half>(D, rows, paged); }
}  // namespace kvd
