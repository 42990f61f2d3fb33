// kvd_prefix_tc5.cuh -- the shared-prefix kernel of 16-bit caches on tcgen05.
//
// One CTA per SM works on up to two 128-row blocks of a KV head at once (A and
// B), against key tiles of 128:
//   * warp 8, the producer: Q blocks by a 4-D TMA box (64 columns x gN rows x 1
//     head x seqs sequences: the box gathers the sequences' rows) at a piece's
//     start; K and V tiles by 2-D TMA boxes of 64 keys x 128 bytes (a box never
//     leaves a page) into a ring whose slots hold one K or one V tile each;
//   * warp 9, the issuer: one thread issues S_X = Q_X . K^T (128 x 128 x D) and
//     O_X += P_X . V (128 x D x 128) for X = A, B; before a last, partial tile's
//     P . V the warp zeroes the value rows past the prefix (a zero weight times
//     a stale NaN is NaN);
//   * warps 0-3 and 4-7, the softmax warps of A and B: thread r owns row r
//     (tensor-memory lane r): running max and sum in registers, weights P back
//     into tensor memory as 16-bit pairs over the columns of S, O rescaled there
//     when the max grows by more than 2^8.
// While the softmax warps of one block work, the tensor core runs the other
// block's products.  Tensor memory: S_A, S_B of 128 columns (P_X over the first
// 64 of S_X), O_A, O_B of D columns: all 512 for D = 128.
//
// S_X of the next tile overwrites P_X, so the issuer waits for P_X . V to
// complete first (its commit on pv_done): it issues both blocks' P . V, then both
// blocks' next S, so that the tensor core has work during that wait.  The O that
// a softmax warp rescales is stable then: S_X(j) is issued after P_X . V(j - 1)
// completed, and P_X . V(j) waits for the warp's own arrival.
//
// Every mbarrier is waited for phase by phase in order; every wait is bounded
// and ends when another warp has given up; a CTA that gave up drains its copies
// and products before it frees the tensor memory.
#pragma once

#include "kvd_attention_tc5.cuh"
#include "kvd_prefix.cuh"

namespace kvd {

template <int D> struct PrefixTc5Shape {
    static constexpr int kTK = 128;
    static constexpr int kBoxes = D / 64;               // 128-byte column boxes of a row
    static constexpr int kBoxBytes = kTK * 128;         // one column box of a tile (or Q block)
    static constexpr int kTileBytes = kBoxes * kBoxBytes;
    static constexpr int kSlots = D == 128 ? 5 : 6;     // ring slots (a K or a V tile each)
    static constexpr int kThreads = 320;
    static constexpr int kTmemCols = 512;
    static constexpr int kTmemS = 0, kTmemO = 256;      // S_X at 128 X; O_X at 256 + D X
    static constexpr int kQOff = kSlots * kTileBytes;
    static constexpr int kBarOff = kQOff + 2 * kTileBytes;
    // full[kSlots], empty[kSlots], q_full, q_empty, s_full[2], p_full[2], pv_done[2], mma_done
    static constexpr int kNumBars = 2 * kSlots + 9;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // tensor-memory base, abort flag
    static constexpr int kSmemBytes = kMiscOff + 16;
    static_assert(D == 64 || D == 128, "head dim");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    // two CTAs (of any tcgen05 kernel here) on one SM would share its tensor memory
    static_assert(2 * kSmemBytes > 227 * 1024, "one CTA per SM");
};

// 4-D tiled TMA load (see tma_load_2d).
__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int x, int y, int z, int w, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}
// 2-D tiled TMA load without an L2 policy: other CTAs read the same tile.
__device__ __forceinline__ void tma_load_2d_shared(void *dst, const void *tmap, int x, int y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

template <typename T, int D, bool kPaged>
__global__ void __launch_bounds__(320, 1)
    prefix_tc5_kernel(const PrefixArgs a, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q)
{
    using S = PrefixTc5Shape<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr float kRescaleThreshold = 8.0f;
    const float kNegInf = __int_as_float(0xff800000);
    extern __shared__ __align__(1024) unsigned char smem_prefix[];
    unsigned char *smem = smem_prefix;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kBarOff);
    uint64_t *empty = full + S::kSlots;
    uint64_t *q_full = empty + S::kSlots, *q_empty = q_full + 1;
    uint64_t *s_full = q_full + 2, *p_full = s_full + 2, *pv_done = p_full + 2, *mma_done = pv_done + 2;
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + S::kMiscOff);
    volatile uint32_t *abort = misc + 1;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

    // The swizzled boxes need 1024-byte-aligned shared memory (checked; every
    // thread takes the same branch, before any barrier or allocation).
    if ((smem_addr(smem) & 1023u) != 0) {
        if (tid == 0) raise_error(a.err_word, KVD_DEVERR_INTERNAL);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < S::kSlots; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(mma_done, 1);
        misc[1] = 0u;
        fence_mbar_init();
    }
    if (warp == 9) {
        tc5_alloc(&misc[0], S::kTmemCols);
        tc5_relinquish();
    }
    // No griddepcontrol.wait yet: this kernel's CTAs start once every CTA of the
    // launch before it (the same call's attention over the own caches) has
    // passed its own wait for everything older, and that launch writes nothing
    // that is read or written here.
    tc5_fence_before();
    __syncthreads();
    tc5_fence_after();
    const uint32_t tmem = misc[0];
    int lo, hi;
    prefix_range(a, &lo, &hi);
    const int u_lo = lo / a.n_tiles, k_lo = lo % a.n_tiles;  // first unit and tile

    if (warp == 8) {
        // ---- producer ----
        if (lane == 0) {
            int fills = 0, q_loads = 0;
            bool dead = false;
            // the next ring slot, free
            auto take = [&]() -> int {
                const int s = fills % S::kSlots;
                if (fills >= S::kSlots && !tc5_wait(&empty[s], (uint32_t)(fills / S::kSlots - 1) & 1u, abort)) return -1;
                ++fills;
                return s;
            };
            auto load_tile = [&](const CUtensorMap *map, int h, int tile, uint32_t extra) -> bool {
                const int s = take();
                if (s < 0) return false;
                unsigned char *dst = smem + s * S::kTileBytes;
                mbar_arrive_expect_tx(&full[s], (uint32_t)S::kTileBytes + extra);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    // (a half past the prefix loads rows that are masked: the first half's again)
                    int key = tile * S::kTK + half * 64;
                    if (key >= a.S) key = tile * S::kTK;
                    int y;
                    if constexpr (kPaged) {
                        int page = __ldg(a.table + (key >> a.page_shift));
                        if ((unsigned)page >= (unsigned)a.num_pages) {  // never read outside the pool
                            raise_error(a.err_word, KVD_DEVERR_PAGE);
                            page = 0;
                        }
                        y = ((page * a.H_kv + h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
                    } else {
                        y = h * a.S_max + key;
                    }
#pragma unroll
                    for (int bx = 0; bx < S::kBoxes; ++bx)
                        tma_load_2d_shared(dst + bx * S::kBoxBytes + half * 64 * 128, map, bx * 64, y, &full[s]);
                }
                return true;
            };
            int u = u_lo, k = k_lo;
            for (int t = lo; t < hi && !dead; ++t) {
                const int h = u / a.units_per_head;
                if (t == lo || k == 0) {  // a piece starts: its Q blocks
                    if (q_loads > 0 && !tc5_wait(q_empty, (uint32_t)(q_loads - 1) & 1u, abort)) {
                        dead = true;
                        break;
                    }
                    const int b0 = (u % a.units_per_head) * a.unit_blocks;
                    const int nb = min(a.unit_blocks, a.blocks - b0);
                    const uint32_t box = (uint32_t)(a.row_blocks == 1 ? a.seqs * a.gN : kPrefixBlock) * 128u;
                    mbar_arrive_expect_tx(q_full, box * (uint32_t)(nb * S::kBoxes));
                    for (int x = 0; x < nb; ++x) {
                        const int2 o = prefix_block_origin(a, b0 + x);
#pragma unroll
                        for (int bx = 0; bx < S::kBoxes; ++bx)
                            tma_load_4d(smem + S::kQOff + x * S::kTileBytes + bx * S::kBoxBytes, &tm_q, bx * 64, o.y, h, o.x,
                                        q_full);
                    }
                    ++q_loads;
                }
                uint32_t extra = 0u;
#ifdef KVD_TIMEOUT_TEST
                if ((a.flags & kPrefixTestStall) && t == lo) extra = 16u;  // a stage that never completes
#endif
                dead = !load_tile(&tm_k, h, k, extra) || !load_tile(&tm_v, h, k, 0u);
                if (++k == a.n_tiles) {
                    k = 0;
                    ++u;
                }
            }
            if (dead) {
                *abort = 1u;
                raise_error(a.err_word, KVD_DEVERR_TIMEOUT);
                // copies still in flight land before the CTA exits (one deadline)
                const uint64_t t0 = global_timer_ns();
                for (int f = max(0, fills - S::kSlots); f < fills; ++f)
                    while (!mbar_try_wait(&full[f % S::kSlots], (uint32_t)(f / S::kSlots) & 1u) &&
                           global_timer_ns() - t0 < kDrainLimitNs) {
                    }
                if (q_loads > 0)
                    while (!mbar_try_wait(q_full, (uint32_t)(q_loads - 1) & 1u) && global_timer_ns() - t0 < kDrainLimitNs) {
                    }
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        // ---- issuer ----
        constexpr uint32_t kIdescS = tc5_idesc<kBf16>(128, S::kTK, false, false);
        constexpr uint32_t kIdescO = tc5_idesc<kBf16>(128, D, false, true);
        const uint32_t ring = smem_addr(smem), qbuf = smem_addr(smem + S::kQOff);
        bool dead = false;
        // waits by lane 0, decided for the warp
        auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
            int ok = 1;
            if (lane == 0) ok = tc5_wait(bar, parity & 1u, abort) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) dead = true;
            return ok != 0;
        };
        auto issue_s = [&](int x, uint32_t kt) {
            if (lane == 0) {
                tc5_fence_after();
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc5_mma_f16(tmem + S::kTmemS + x * 128,
                                tc5_desc(qbuf + x * S::kTileBytes + (ks >> 2) * S::kBoxBytes + (ks & 3) * 32, 0u, 1024u),
                                tc5_desc(kt + (ks >> 2) * S::kBoxBytes + (ks & 3) * 32, 0u, 1024u), kIdescS,
                                ks > 0 ? 1u : 0u);
                tc5_commit(&s_full[x]);
            }
        };
        auto issue_pv = [&](int x, uint32_t vt, bool first) {
            if (lane == 0) {
                tc5_fence_after();
#pragma unroll
                for (int ks = 0; ks < S::kTK / 16; ++ks)
                    tc5_mma_f16_ts(tmem + S::kTmemO + x * D, tmem + S::kTmemS + x * 128 + ks * 8,
                                   tc5_desc(vt + ks * 16 * 128, (uint32_t)S::kBoxBytes, 1024u), kIdescO,
                                   (ks > 0 || !first) ? 1u : 0u);
                tc5_commit(&pv_done[x]);
            }
        };
        int u = u_lo, k = k_lo, f = 0;  // f: ring fills consumed (K of this tile is fill f)
        int pieces = 0;
        uint32_t n_s[2] = {0u, 0u};     // tiles of each block so far (phases of its barriers)
        bool have_s = false;            // S of tile t is issued already
        for (int t = lo; t < hi && !dead; ++t) {
            const int nb = min(a.unit_blocks, a.blocks - (u % a.units_per_head) * a.unit_blocks);
            const bool first = t == lo || k == 0;
            const bool last = t == hi - 1 || k == a.n_tiles - 1;
            if (!have_s) {
                if (!wait(q_full, (uint32_t)pieces)) break;
                ++pieces;
                if (!wait(&full[f % S::kSlots], (uint32_t)(f / S::kSlots))) break;
                // (S_X lies over the previous piece's last P_X)
                for (int x = 0; x < nb && !dead; ++x)
                    if (n_s[x] > 0u) wait(&pv_done[x], n_s[x] - 1u);
                if (dead) break;
                for (int x = 0; x < nb; ++x) issue_s(x, ring + (f % S::kSlots) * S::kTileBytes);
                if (lane == 0) {
                    tc5_commit(&empty[f % S::kSlots]);
                    if (last) tc5_commit(q_empty);
                }
            }
            const int fv = f + 1, sv = fv % S::kSlots;
            if (!wait(&full[sv], (uint32_t)(fv / S::kSlots))) break;
            const uint32_t vt = ring + sv * S::kTileBytes;
            const int nk = a.S - k * S::kTK;
            if (nk < S::kTK) {  // value rows past the prefix: zero
                for (int idx = lane; idx < (S::kTK - nk) * (D / 8); idx += 32) {
                    const int r = nk + idx / (D / 8), c = idx % (D / 8);
                    const uint32_t lin = vt + (c >> 3) * S::kBoxBytes + r * 128 + ((c & 7) << 4);
                    sts128(lin ^ ((lin >> 3) & 0x70u), make_uint4(0u, 0u, 0u, 0u));
                }
                fence_proxy_async_shared();
                __syncwarp();
            }
            for (int x = 0; x < nb && !dead; ++x) {
                if (!wait(&p_full[x], n_s[x])) break;
                issue_pv(x, vt, first);
            }
            if (dead) break;
            if (lane == 0) tc5_commit(&empty[sv]);
            have_s = !last;
            if (!last) {  // the next tile's S, each block's once its P . V is complete
                const int fk = f + 2, sk = fk % S::kSlots;
                if (!wait(&full[sk], (uint32_t)(fk / S::kSlots))) break;
                const bool next_last = t + 1 == hi - 1 || k + 1 == a.n_tiles - 1;
                for (int x = 0; x < nb && !dead; ++x) {
                    if (!wait(&pv_done[x], n_s[x])) break;
                    issue_s(x, ring + sk * S::kTileBytes);
                }
                if (dead) break;
                if (lane == 0) {
                    tc5_commit(&empty[sk]);
                    if (next_last) tc5_commit(q_empty);
                }
            }
            for (int x = 0; x < nb; ++x) ++n_s[x];
            f += 2;
            if (++k == a.n_tiles) {
                k = 0;
                ++u;
            }
        }
        if (lane == 0) {
            if (dead) {
                *abort = 1u;
                raise_error(a.err_word, KVD_DEVERR_TIMEOUT);
            }
            tc5_commit(mma_done);  // this thread's products complete before the tensor memory is freed
            mbar_wait_drain(mma_done, 0u);
        }
        __syncwarp();
    } else {
        // ---- softmax warps: block x, row r ----
        const int x = warp / 4, r = tid % 128;
        const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t t_s = tmem + lanes + S::kTmemS + x * 128, t_o = tmem + lanes + S::kTmemO + x * D;
        float m_run = kNegInf, l_run = 0.f;
        uint32_t n_s = 0u;
        bool dead = false;
        auto warp_wait = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, tc5_wait(bar, parity & 1u, abort));
        };
        int u = u_lo, k = k_lo;
        for (int t = lo; t < hi; ++t) {
            const int b0 = (u % a.units_per_head) * a.unit_blocks;
            const bool first = t == lo || k == 0;
            const bool last = t == hi - 1 || k == a.n_tiles - 1;
            if (b0 + x < a.blocks) {
                if (first) {
                    m_run = kNegInf;
                    l_run = 0.f;
                }
                if (!warp_wait(&s_full[x], n_s)) {
                    dead = true;
                    break;
                }
                tc5_fence_after();
                uint32_t s0[64], s1[64];
                tc5_ld64(t_s, s0);
                tc5_ld64(t_s + 64, s1);
                const int nk = a.S - k * S::kTK;
                if (nk < S::kTK) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        if (c >= nk) s0[c] = 0xff800000u;  // -inf
                        if (64 + c >= nk) s1[c] = 0xff800000u;
                    }
                }
                float mx[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mx[i] = fmaxf(__uint_as_float(s0[i]), __uint_as_float(s1[i]));
#pragma unroll
                for (int c = 8; c < 64; ++c) mx[c & 7] = fmaxf(mx[c & 7], fmaxf(__uint_as_float(s0[c]), __uint_as_float(s1[c])));
                const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                        fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * a.qscale;
                float alpha = 1.f;
                bool rescale = false;
                if (top > m_run + kRescaleThreshold) {
                    if (!first) {
                        alpha = fast_exp2(m_run - top);
                        rescale = true;
                    }
                    m_run = top;
                }
                if (__any_sync(0xffffffffu, rescale)) {  // (rows that keep their max scale by 1)
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tc5_ld32(t_o + c0, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tc5_st32(t_o + c0, o);
                    }
                }
                const float nmu = (m_run == kNegInf) ? 0.f : -m_run;
                float l8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) l8[i] = 0.f;
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float p0 = fast_exp2(fmaf(__uint_as_float(s0[2 * c]), a.qscale, nmu));
                    const float p1 = fast_exp2(fmaf(__uint_as_float(s0[2 * c + 1]), a.qscale, nmu));
                    l8[c & 7] += p0 + p1;
                    pk[c] = pack_pair<T>(p0, p1);
                }
                tc5_st32(t_s, pk);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float p0 = fast_exp2(fmaf(__uint_as_float(s1[2 * c]), a.qscale, nmu));
                    const float p1 = fast_exp2(fmaf(__uint_as_float(s1[2 * c + 1]), a.qscale, nmu));
                    l8[c & 7] += p0 + p1;
                    pk[c] = pack_pair<T>(p0, p1);
                }
                tc5_st32(t_s + 32, pk);
                l_run = l_run * alpha + (((l8[0] + l8[1]) + (l8[2] + l8[3])) + ((l8[4] + l8[5]) + (l8[6] + l8[7])));
                tc5_fence_before();
                mbar_arrive(&p_full[x]);
                if (last) {
                    // ---- end of a piece: its (o, m, l) ----
                    if (!warp_wait(&pv_done[x], n_s)) {
                        dead = true;
                        break;
                    }
                    tc5_fence_after();
                    const size_t slot = (size_t)(u + (int)blockIdx.x);
                    const int sr = x * kPrefixBlock + r;
                    float4 *po = reinterpret_cast<float4 *>(a.part) + slot * (D / 4) * a.slot_rows + sr;
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tc5_ld32(t_o + c0, o);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            __stcg(po + (size_t)((c0 + i) / 4) * a.slot_rows,
                                   make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                                               __uint_as_float(o[i + 3])));
                    }
                    a.part_ml[slot * 2 * a.slot_rows + sr] = m_run;
                    a.part_ml[(slot * 2 + 1) * a.slot_rows + sr] = l_run;
                    tc5_fence_before();  // (the next arrive on p_full orders these reads before O is overwritten)
                }
                ++n_s;
            }
            if (++k == a.n_tiles) {
                k = 0;
                ++u;
            }
        }
        if (dead) {
            *abort = 1u;
            raise_error(a.err_word, KVD_DEVERR_TIMEOUT);
        }
    }

    tc5_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc5_fence_after();
        tc5_dealloc(tmem, S::kTmemCols);
    }
    // This grid completes only after the launch before it has: the join, which
    // waits for this grid, may read what both wrote.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename T> bool pick_prefix_tc5(int D, bool paged, PrefixVariant *v)
{
    if (D != 64 && D != 128) return false;
    if (D == 64) {
        v->fn = paged ? reinterpret_cast<const void *>(&prefix_tc5_kernel<T, 64, true>)
                      : reinterpret_cast<const void *>(&prefix_tc5_kernel<T, 64, false>);
        v->join_fn = reinterpret_cast<const void *>(&prefix_join_kernel<T, 64>);
        v->smem_bytes = PrefixTc5Shape<64>::kSmemBytes;
    } else {
        v->fn = paged ? reinterpret_cast<const void *>(&prefix_tc5_kernel<T, 128, true>)
                      : reinterpret_cast<const void *>(&prefix_tc5_kernel<T, 128, false>);
        v->join_fn = reinterpret_cast<const void *>(&prefix_join_kernel<T, 128>);
        v->smem_bytes = PrefixTc5Shape<128>::kSmemBytes;
    }
    v->threads = PrefixTc5Shape<128>::kThreads;
    v->tile_keys = PrefixTc5Shape<128>::kTK;
    v->join_grid_y = D / 4 / (4 * kJoinCols);
    v->tma = true;
    return true;
}

}  // namespace kvd
