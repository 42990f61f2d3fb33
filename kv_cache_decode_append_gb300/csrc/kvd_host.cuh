// kvd_host.cuh -- host helpers of the entry points, shared by their translation
// units (defined in kvd_api.cu).
#pragma once

#include <cuda.h>
#include <stddef.h>
#include <stdint.h>

#include "kvd.h"

namespace kvd {

// A paged cache's block table and pool geometry.
struct PagedCache {
    const int32_t *block_table;
    int page_size, max_pages, num_pages;
};

// Checks of the paged geometry; on success *T_max = max_pages * page_size.
kvd_status check_paged(const PagedCache &pc, int *T_max, int *page_shift);

// SMs of the current device.
kvd_status current_sm_count(int *sms);

int elem_bytes(kvd_dtype dt);  // 0: unknown
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// A tensor map of 16-bit elements with the 128-byte swizzle (strides: bytes,
// rank - 1 of them; box: elements, its rows 128 bytes).
kvd_status encode_map_16bit(CUtensorMap *map, const void *base, kvd_dtype dtype, int rank, const uint64_t *dims,
                            const uint64_t *strides, const uint32_t *box);

// Opts `fn` into `smem` bytes of dynamic shared memory on the current device.
kvd_status kernel_ready(const void *fn, int threads, int smem);

// The attention kernels leaving row states instead of an output (for a join):
// where their workspace keeps them, and the launch itself.  Arguments and
// checks of kvd_decode_attention / kvd_paged_decode_attention; the workspace
// needs no initial contents.
struct RowStatePlan {
    int rb, n_rowblocks, prow;  // rows per block, blocks per head, rows per piece slot
    int pair_grid;              // > 0: the pair kernel's CTAs (rb 256) ...
    int max_splits, cta_tiles;  // ... max_splits > 0: the streaming kernel's slots per head, and their tiles, instead
    int grid;                   // its CTAs
    size_t part_off, seg_off, state_off, bytes;
};
kvd_status row_state_plan(int B, int H_q, int H_kv, int D, int N, int max_past_len, kvd_dtype dtype, bool paged,
                          RowStatePlan *plan);
kvd_status row_state_check(const void *q, const void *k_cache, const void *v_cache, const int32_t *past_len, int B,
                           int H_q, int H_kv, int T_max, int D, int N, int max_past_len, kvd_dtype dtype,
                           const PagedCache *paged);
kvd_status row_state_launch(const void *q, const void *k_cache, const void *v_cache, const int32_t *past_len, int B,
                            int H_q, int H_kv, int T_max, int D, int N, int max_past_len, float scale,
                            kvd_dtype dtype, const PagedCache *paged, void *workspace, size_t workspace_bytes,
                            uint32_t *err_word, void *stream);

#ifdef KVD_TIMEOUT_TEST
extern int g_test_stall;  // test builds: plant a stall in the next launches
#endif

}  // namespace kvd
