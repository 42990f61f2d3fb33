// kvd_host.cuh -- host helpers of the entry points, shared by their translation
// units (defined in kvd_api.cu).
#pragma once

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

}  // namespace kvd
