// kvd_prefix_api.cu -- the entry points of attention over a shared prefix:
// checks, the split of the prefix, and the call's three launches (kvd_prefix.cuh).
#include <math.h>

#include <algorithm>

#include "kvd_host.cuh"
#include "kvd_prefix.cuh"

namespace kvd {
namespace {

bool pick_prefix(kvd_dtype dtype, int D, bool paged, PrefixVariant *v)
{
    switch (dtype) {
    case KVD_F32: return prefix_variant_f32(D, paged, v);
    case KVD_BF16: return prefix_variant_bf16(D, paged, v);
    case KVD_F16: return prefix_variant_f16(D, paged, v);
    default: return false;
    }
}

struct PrefixPlan {
    RowStatePlan own;
    PrefixVariant v;
    int seqs, row_blocks, blocks, unit_blocks, units_per_head, n_units, n_tiles, grid, slot_rows;
    size_t ml_off, part_off, bytes;
};

kvd_status make_prefix_plan(int B, int H_q, int H_kv, int D, int N, int S, int max_past_len, kvd_dtype dtype, bool paged,
                            PrefixPlan *pl)
{
    if (S < 0) return KVD_ERR_INVALID_ARG;
    kvd_status st = row_state_plan(B, H_q, H_kv, D, N, max_past_len, dtype, paged, &pl->own);
    if (st != KVD_OK) return st;
    if (!pick_prefix(dtype, D, paged, &pl->v)) return KVD_ERR_UNSUPPORTED;
    int sms = 0;
    if ((st = current_sm_count(&sms)) != KVD_OK) return st;
    const int gN = H_q / H_kv * N;
    pl->seqs = gN <= kPrefixBlock ? kPrefixBlock / gN : 1;
    pl->row_blocks = gN <= kPrefixBlock ? 1 : (gN + kPrefixBlock - 1) / kPrefixBlock;
    const long long blocks = pl->row_blocks == 1 ? ((long long)B + pl->seqs - 1) / pl->seqs : (long long)B * pl->row_blocks;
    pl->unit_blocks = pl->v.tma && blocks > 1 ? 2 : 1;
    const long long per_head = (blocks + pl->unit_blocks - 1) / pl->unit_blocks;
    pl->n_tiles = (S + pl->v.tile_keys - 1) / pl->v.tile_keys;
    const long long n = (long long)H_kv * per_head * std::max(pl->n_tiles, 1);
    if (n > 0x7fffffffLL || (long long)H_kv * blocks * 4 > 0x7fffffffLL) return KVD_ERR_UNSUPPORTED;
    pl->blocks = (int)blocks;
    pl->units_per_head = (int)per_head;
    pl->n_units = (int)(H_kv * per_head);
    pl->grid = (int)std::min<long long>(sms, n);
    pl->slot_rows = pl->unit_blocks * kPrefixBlock;
    const size_t slots = pl->n_tiles > 0 ? (size_t)pl->n_units + pl->grid - 1 : 0;
    size_t off = round_up(pl->own.bytes, 256);
    pl->ml_off = off;
    off += round_up(slots * 2 * pl->slot_rows * sizeof(float), 256);
    pl->part_off = off;
    off += round_up(slots * pl->slot_rows * D * sizeof(float), 256);
    pl->bytes = off;
    return KVD_OK;
}

kvd_status prefix_launch(const void *q, const void *k_prefix, const void *v_prefix, const int32_t *prefix_table,
                         const void *k_cache, const void *v_cache, void *out, const int32_t *past_len, int B, int H_q,
                         int H_kv, int S_max, int T_max, int D, int N, int S, int max_past_len, float scale,
                         kvd_dtype dtype, const PagedCache *paged, void *workspace, size_t workspace_bytes,
                         uint32_t *err_word, void *stream)
{
    kvd_status st = row_state_check(q, k_cache, v_cache, past_len, B, H_q, H_kv, T_max, D, N, max_past_len, dtype, paged);
    if (st != KVD_OK) return st;
    if (!out || !aligned16(out) || S < 0) return KVD_ERR_INVALID_ARG;
    int page_shift = 0;
    if (paged != nullptr) {
        if ((st = check_paged(*paged, &T_max, &page_shift)) != KVD_OK) return st;
        if (S > 0 && (!prefix_table || (reinterpret_cast<uintptr_t>(prefix_table) & 3u) != 0)) return KVD_ERR_INVALID_ARG;
        if (((long long)S + paged->page_size - 1) / paged->page_size > paged->num_pages) return KVD_ERR_CAPACITY;
    } else if (S > 0) {
        if (!k_prefix || !v_prefix || !aligned16(k_prefix) || !aligned16(v_prefix)) return KVD_ERR_INVALID_ARG;
        if (S > S_max) return KVD_ERR_CAPACITY;
    }
    if (B == 0) return KVD_OK;

    PrefixPlan pl;
    if ((st = make_prefix_plan(B, H_q, H_kv, D, N, S, max_past_len, dtype, paged != nullptr, &pl)) != KVD_OK) return st;
    if (workspace == nullptr || workspace_bytes < pl.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return KVD_ERR_WORKSPACE;
    const int gN = H_q / H_kv * N;
    if (pl.v.tma && (long long)S + 128 > 0x7fffffffLL) return KVD_ERR_UNSUPPORTED;  // 32-bit box coordinates

    char *ws = static_cast<char *>(workspace);
    PrefixArgs a = {};
    a.q = q;
    a.k = k_prefix;
    a.v = v_prefix;
    a.table = prefix_table;
    a.part = reinterpret_cast<float *>(ws + pl.part_off);
    a.part_ml = reinterpret_cast<float *>(ws + pl.ml_off);
    a.err_word = err_word;
    a.B = B;
    a.H_kv = H_kv;
    a.gN = gN;
    a.S = S;
    a.S_max = S_max;
    a.seqs = pl.seqs;
    a.row_blocks = pl.row_blocks;
    a.blocks = pl.blocks;
    a.unit_blocks = pl.unit_blocks;
    a.units_per_head = pl.units_per_head;
    a.n_units = pl.n_units;
    a.n_tiles = pl.n_tiles;
    a.slot_rows = pl.slot_rows;
    a.page_shift = page_shift;
    a.num_pages = paged != nullptr ? paged->num_pages : 0;
    a.qscale = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * kLog2e;
#ifdef KVD_TIMEOUT_TEST
    if (g_test_stall) a.flags = kArgTestStall;
#endif
    // (all that can be refused comes before the first launch)
    alignas(64) CUtensorMap tmk, tmv, tmv_last, tmq;
    if (S > 0) {
        if ((st = kernel_ready(pl.v.fn, pl.v.threads, pl.v.smem_bytes)) != KVD_OK) return st;
        if (pl.v.tma) {
            // (column, row, head, page) of the prefix; the rows end where it ends,
            // so that TMA fills what lies past it with zeros
            const uint64_t per_page = paged != nullptr ? (uint64_t)paged->page_size : (uint64_t)S_max;
            const uint64_t strides[3] = {(uint64_t)D * 2, per_page * D * 2, per_page * D * 2 * H_kv};
            const uint32_t box[4] = {64, 64, 1, 1};
            uint64_t dims[4] = {(uint64_t)D, paged != nullptr ? per_page : (uint64_t)S, (uint64_t)H_kv,
                                paged != nullptr ? (uint64_t)paged->num_pages : 1u};
            if ((st = encode_map_16bit(&tmk, k_prefix, dtype, 4, dims, strides, box)) != KVD_OK) return st;
            if ((st = encode_map_16bit(&tmv, v_prefix, dtype, 4, dims, strides, box)) != KVD_OK) return st;
            if (paged != nullptr) dims[1] = (uint64_t)((S - 1) % paged->page_size + 1);
            if ((st = encode_map_16bit(&tmv_last, v_prefix, dtype, 4, dims, strides, box)) != KVD_OK) return st;
            const uint64_t qdims[4] = {(uint64_t)D, (uint64_t)gN, (uint64_t)H_kv, (uint64_t)B};
            const uint64_t qstrides[3] = {(uint64_t)D * 2, (uint64_t)gN * D * 2, (uint64_t)H_kv * gN * D * 2};
            const uint32_t qbox[4] = {64, (uint32_t)std::min(gN, kPrefixBlock), 1, (uint32_t)pl.seqs};
            if ((st = encode_map_16bit(&tmq, q, dtype, 4, qdims, qstrides, qbox)) != KVD_OK) return st;
        }
    }

    // 1. the sequences' own keys
    if ((st = row_state_launch(q, k_cache, v_cache, past_len, B, H_q, H_kv, T_max, D, N, max_past_len, scale, dtype, paged,
                               ws, pl.own.bytes, err_word, stream)) != KVD_OK)
        return st;

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // 2. the prefix
    if (S > 0) {
        cfg.gridDim = dim3((unsigned)pl.grid);
        cfg.blockDim = dim3((unsigned)pl.v.threads);
        cfg.dynamicSmemBytes = (size_t)pl.v.smem_bytes;
        void *args[] = {&a, &tmk, &tmv, &tmv_last, &tmq};
        if (cudaLaunchKernelExC(&cfg, pl.v.fn, args) != cudaSuccess) return KVD_ERR_CUDA;
    }
    // 3. the join
    RowStateArgs s = {};
    s.state = reinterpret_cast<const float *>(ws + pl.own.state_off);
    s.part = reinterpret_cast<const float *>(ws + pl.own.part_off);
    s.seg = reinterpret_cast<const int2 *>(ws + pl.own.seg_off);
    s.past_len = past_len;
    s.rb = pl.own.rb;
    s.n_rowblocks = pl.own.n_rowblocks;
    s.prow = pl.own.prow;
    s.pair_grid = pl.own.pair_grid;
    s.max_splits = pl.own.max_splits;
    s.cta_tiles = pl.own.cta_tiles;
    s.T_max = T_max;
    s.max_past_len = max_past_len;
    s.N = N;
    s.grid = pl.grid;
    s.own_grid = pl.own.grid;
    cfg.gridDim = dim3((unsigned)(H_kv * pl.blocks * (kPrefixBlock / 32)), (unsigned)pl.v.join_grid_y);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    void *args[] = {&a, &s, &out};
    return cudaLaunchKernelExC(&cfg, pl.v.join_fn, args) == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" {

size_t kvd_shared_prefix_workspace_bytes(int B, int H_q, int H_kv, int D, int N, int prefix_len, int max_past_len,
                                         kvd_dtype dtype)
{
    PrefixPlan a, b;  // (one size for both cache layouts)
    if (make_prefix_plan(B, H_q, H_kv, D, N, prefix_len, max_past_len, dtype, false, &a) != KVD_OK ||
        make_prefix_plan(B, H_q, H_kv, D, N, prefix_len, max_past_len, dtype, true, &b) != KVD_OK)
        return 0;
    return std::max(a.bytes, b.bytes);
}

kvd_status kvd_shared_prefix_attention(const void *q, const void *k_prefix, const void *v_prefix, const void *k_cache,
                                       const void *v_cache, void *out, const int32_t *past_len, int B, int H_q,
                                       int H_kv, int S_max, int T_max, int D, int N, int prefix_len, int max_past_len,
                                       float scale, kvd_dtype dtype, void *workspace, size_t workspace_bytes,
                                       uint32_t *err_word, void *stream)
{
    return prefix_launch(q, k_prefix, v_prefix, nullptr, k_cache, v_cache, out, past_len, B, H_q, H_kv, S_max, T_max, D, N,
                         prefix_len, max_past_len, scale, dtype, nullptr, workspace, workspace_bytes, err_word, stream);
}

kvd_status kvd_paged_shared_prefix_attention(const void *q, const void *k_pages, const void *v_pages, void *out,
                                             const int32_t *prefix_table, const int32_t *block_table,
                                             const int32_t *past_len, int B, int H_q, int H_kv, int D, int N,
                                             int page_size, int max_pages, int num_pages, int prefix_len,
                                             int max_past_len, float scale, kvd_dtype dtype, void *workspace,
                                             size_t workspace_bytes, uint32_t *err_word, void *stream)
{
    const PagedCache pc{block_table, page_size, max_pages, num_pages};
    return prefix_launch(q, k_pages, v_pages, prefix_table, k_pages, v_pages, out, past_len, B, H_q, H_kv, 0, 0, D, N,
                         prefix_len, max_past_len, scale, dtype, &pc, workspace, workspace_bytes, err_word, stream);
}

}  // extern "C"
