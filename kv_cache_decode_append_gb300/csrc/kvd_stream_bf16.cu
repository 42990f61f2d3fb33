// Instantiates the bf16 streaming attention kernels with modified scores.
#include "kvd_attention_stream.cuh"

namespace kvd {
const void *stream_kernel_bf16(int D, int rows, bool paged) { return pick_stream_kernel<__nv_bfloat16>(D, rows, paged); }
}  // namespace kvd
