// kvd_prefix_tc5.cuh -- the shared-prefix kernel of 16-bit caches on tcgen05.
//
// One CTA per SM works on up to two 128-row blocks of a KV head at once (A and
// B), against key tiles of 128:
//   * warp 8, the producer: Q blocks by a 4-D TMA box (64 columns x gN rows x 1
//     head x seqs sequences: the box gathers the sequences' rows) at a piece's
//     start; K and V tiles by 4-D TMA boxes of 64 keys x 128 bytes (a box never
//     leaves a page) into a ring whose slots hold one K or one V tile each.
//     Value rows past the prefix must be zeros (a zero weight times a stale NaN
//     is NaN): the maps end at the prefix (its last page has a map of its own),
//     and TMA fills what lies outside a map with zeros;
//   * warp 9, the issuer: one thread issues S_X = Q_X . K^T (128 x 128 x D) and
//     O_X += P_X . V (128 x D x 128) for X = A, B;
//   * warps 0-3 and 4-7, the softmax warps of A and B: thread r owns row r
//     (tensor-memory lane r): running max and sum in registers, weights P back
//     into tensor memory as 16-bit pairs over the columns of S, O rescaled there
//     when the max grows by more than 2^8.
// While the softmax warps of one block work, the tensor core runs the other
// block's products.  Tensor memory: S_A, S_B of 128 columns (P_X over the first
// 64 of S_X), O_A, O_B of D columns: all 512 for D = 128.
//
// A block's chain is S -> softmax -> P . V -> S of the next tile, which
// overwrites P_X: the issuer waits for P_X . V to complete first (its commit on
// pv_done).  The O that a softmax warp rescales is stable then: S_X(j) is issued
// after P_X . V(j - 1) completed, and P_X . V(j) waits for the warp's arrival.
// What bounds the loop is shared memory: S reads 8 KB of operands per 64 cycles
// of the tensor core, all that shared memory delivers, P . V half, TMA writes the
// tiles; a barrier tested meanwhile takes 100 cycles and more.  So the issuer is
// one thread that blocks on the barriers in their expected order.  Measured at
// 16384 keys, 8 KV heads of 512 rows: 36 us so; 39 us with an issuer per block
// (their products take turns and both come late), 40 us with one that tests
// both blocks' barriers in turn, 49 us with whole-warp waits.
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

// 4-D tiled TMA load (see tma_load_2d), without an L2 policy: other CTAs read
// the same tiles.
__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int x, int y, int z, int w, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}
// Bounded wait for phase `parity` of bar that also gives up once *abort is set;
// the clock is read only once the phase is late.
__device__ __forceinline__ bool prefix_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort)
{
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0u) {
            if (*abort != 0u) return false;
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > kWaitLimitNs) return false;
        }
    }
}

// One thread of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  elect.sync _|p, 0xffffffff;\n"
        "  selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(r)
        :
        : "memory");
    return r != 0u;
}

template <typename T, int D, bool kPaged>
__global__ void __launch_bounds__(320, 1)
    prefix_tc5_kernel(const PrefixArgs a, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_v_last,
                      const __grid_constant__ CUtensorMap tm_q)
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
        mbar_init(mma_done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&pv_done[i], 1);
        }
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
                if (fills >= S::kSlots && !prefix_wait(&empty[s], (uint32_t)(fills / S::kSlots - 1) & 1u, abort)) return -1;
                ++fills;
                return s;
            };
            auto load_tile = [&](const CUtensorMap *map, const CUtensorMap *map_last, int h, int tile, uint32_t extra) -> bool {
                const int s = take();
                if (s < 0) return false;
                unsigned char *dst = smem + s * S::kTileBytes;
                mbar_arrive_expect_tx(&full[s], (uint32_t)S::kTileBytes + extra);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int key = tile * S::kTK + half * 64;
                    int row = key, page = 0;  // (row: past the map's end where the half lies past the prefix)
                    const CUtensorMap *m = map;
                    if constexpr (kPaged) {
                        const int last_page = (a.S - 1) >> a.page_shift;
                        const int lp = min(key >> a.page_shift, last_page);
                        row = key - (lp << a.page_shift);
                        if (lp == last_page) m = map_last;
                        page = __ldg(a.table + lp);
                        if ((unsigned)page >= (unsigned)a.num_pages) {  // never read outside the pool
                            raise_error(a.err_word, KVD_DEVERR_PAGE);
                            page = 0;
                        }
                    }
#pragma unroll
                    for (int bx = 0; bx < S::kBoxes; ++bx)
                        tma_load_4d(dst + bx * S::kBoxBytes + half * 64 * 128, m, bx * 64, row, h, page, &full[s]);
                }
                return true;
            };
            int u = u_lo, k = k_lo;
            for (int t = lo; t < hi && !dead; ++t) {
                const int h = u / a.units_per_head;
                if (t == lo || k == 0) {  // a piece starts: its Q blocks
                    if (q_loads > 0 && !prefix_wait(q_empty, (uint32_t)(q_loads - 1) & 1u, abort)) {
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
                dead = !load_tile(&tm_k, &tm_k, h, k, extra) || !load_tile(&tm_v, &tm_v_last, h, k, 0u);
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
        // ---- issuer: one thread ----
        if (elect_one()) {
            constexpr uint32_t kIdescS = tc5_idesc<kBf16>(128, S::kTK, false, false);
            constexpr uint32_t kIdescO = tc5_idesc<kBf16>(128, D, false, true);
            // (a descriptor's address field counts 16 bytes; slots and k-steps add to it)
            const uint64_t desc_q = tc5_desc(smem_addr(smem + S::kQOff), 0u, 1024u);
            const uint64_t desc_k = tc5_desc(smem_addr(smem), 0u, 1024u);
            const uint64_t desc_v = tc5_desc(smem_addr(smem), (uint32_t)S::kBoxBytes, 1024u);
            bool ok = true;
            auto issue_s = [&](int x, int slot) {
                const uint64_t q = desc_q + x * (S::kTileBytes / 16), kd = desc_k + slot * (S::kTileBytes / 16);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const int step = ((ks >> 2) * S::kBoxBytes + (ks & 3) * 32) / 16;
                    tc5_mma_f16(tmem + S::kTmemS + x * 128, q + step, kd + step, kIdescS, ks > 0 ? 1u : 0u);
                }
                tc5_commit(&s_full[x]);
            };
            auto issue_pv = [&](int x, int slot, bool first) {
                const uint64_t vd = desc_v + slot * (S::kTileBytes / 16);
#pragma unroll
                for (int ks = 0; ks < S::kTK / 16; ++ks)
                    tc5_mma_f16_ts(tmem + S::kTmemO + x * D, tmem + S::kTmemS + x * 128 + ks * 8, vd + ks * (16 * 128 / 16),
                                   kIdescO, (ks > 0 || !first) ? 1u : 0u);
                tc5_commit(&pv_done[x]);
            };
            // the ring's next fill (K and V of each tile in turn), as slot and parity
            int slot = 0;
            uint32_t par = 0u;
            auto step = [&]() {
                if (++slot == S::kSlots) {
                    slot = 0;
                    par ^= 1u;
                }
            };
            int u = u_lo, k = k_lo;
            uint32_t pieces = 0u, n0 = 0u, n1 = 0u;  // pieces, and tiles of each block, so far
            bool have_s = false;                     // S of tile t is issued already
            for (int t = lo; t < hi; ++t) {
                const bool two = a.unit_blocks > 1 && (u % a.units_per_head) * 2 + 1 < a.blocks;
                const bool first = t == lo || k == 0;
                const bool last = t == hi - 1 || k == a.n_tiles - 1;
                if (!have_s) {
                    ok = prefix_wait(q_full, pieces & 1u, abort) && prefix_wait(&full[slot], par, abort);
                    ++pieces;
                    // (S_X lies over the previous piece's last P_X)
                    if (ok && n0 > 0u) ok = prefix_wait(&pv_done[0], (n0 - 1u) & 1u, abort);
                    if (ok && two && n1 > 0u) ok = prefix_wait(&pv_done[1], (n1 - 1u) & 1u, abort);
                    if (!ok) break;
                    tc5_fence_after();
                    issue_s(0, slot);
                    if (two) issue_s(1, slot);
                    tc5_commit(&empty[slot]);
                    if (last) tc5_commit(q_empty);
                    step();
                }
                const int vs = slot;
                if (!(ok = prefix_wait(&full[vs], par, abort) && prefix_wait(&p_full[0], n0 & 1u, abort))) break;
                step();
                const int ks = slot;  // the next tile's K
                const bool next_last = t + 1 == hi - 1 || k + 1 == a.n_tiles - 1;
                tc5_fence_after();
                issue_pv(0, vs, first);
                if (!two) tc5_commit(&empty[vs]);
                if (!last) {  // the next tile's S of this block, once its P . V is complete
                    if (!(ok = prefix_wait(&full[ks], par, abort) && prefix_wait(&pv_done[0], n0 & 1u, abort))) break;
                    issue_s(0, ks);
                    if (!two) tc5_commit(&empty[ks]);
                }
                ++n0;
                if (two) {
                    if (!(ok = prefix_wait(&p_full[1], n1 & 1u, abort))) break;
                    tc5_fence_after();
                    issue_pv(1, vs, first);
                    tc5_commit(&empty[vs]);
                    if (!last) {
                        if (!(ok = prefix_wait(&pv_done[1], n1 & 1u, abort))) break;
                        issue_s(1, ks);
                        tc5_commit(&empty[ks]);
                    }
                    ++n1;
                }
                if (!last) {
                    if (next_last) tc5_commit(q_empty);
                    step();
                }
                have_s = !last;
                if (++k == a.n_tiles) {
                    k = 0;
                    ++u;
                }
            }
            if (!ok) {
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
            return __all_sync(0xffffffffu, prefix_wait(bar, parity & 1u, abort));
        };
        int u = u_lo, k = k_lo;
        for (int t = lo; t < hi; ++t) {
            const int b0 = (u % a.units_per_head) * a.unit_blocks;
            const bool first = t == lo || k == 0;
            const bool last = t == hi - 1 || k == a.n_tiles - 1;
            if (b0 + x < a.blocks && x < a.unit_blocks) {
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
                // (four chains of three-input maxima)
                float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                for (int c = 0; c < 64; ++c) mx[c & 3] = max3(mx[c & 3], __uint_as_float(s0[c]), __uint_as_float(s1[c]));
                const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * a.qscale;
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
                // weights 2^(qscale s - m): scale and maximum in one packed FMA,
                // sums as packed pairs in four chains
                const float nmu = (m_run == kNegInf) ? 0.f : -m_run;
                const f32x2 q2 = pack2(a.qscale, a.qscale), nmu2 = pack2(nmu, nmu);
                f32x2 l4[4] = {0ull, 0ull, 0ull, 0ull};
                uint32_t pk[32];
                auto weights = [&](const uint32_t (&s)[64]) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        float y0, y1;
                        unpack2(fma2(pack2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), q2, nmu2), y0, y1);
                        const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
                        l4[c & 3] = add2(l4[c & 3], pack2(p0, p1));
                        pk[c] = pack_pair<T>(p0, p1);
                    }
                };
                weights(s0);
                tc5_st32(t_s, pk);
                weights(s1);
                tc5_st32(t_s + 32, pk);
                float le, lo2;
                unpack2(add2(add2(l4[0], l4[1]), add2(l4[2], l4[3])), le, lo2);
                l_run = l_run * alpha + (le + lo2);
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
    v->join_grid_y = D / 4 / (kJoinThreads / 32);
    v->tma = true;
    return true;
}

}  // namespace kvd
