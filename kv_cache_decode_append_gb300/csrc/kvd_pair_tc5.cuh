// kvd_pair_tc5.cuh -- attention of many query rows over 16-bit caches on
// tcgen05, two 128-row blocks at a time.
//
// One CTA per SM works on up to two 128-row blocks of a KV head at once (A and
// B), against tiles of 128 keys (two halves of 64).  What a CTA works on, which
// keys a tile holds and where results go is a job's (PrefixJob below: a batch's
// rows over one shared prefix; ScoredJob: a sequence's rows with modified
// scores).
//   * warp 8, the producer: Q blocks at a piece's start; K and V tiles by 4-D TMA
//     boxes of 64 keys x 128 bytes (a box never leaves a page) into a ring whose
//     slots hold one K or one V tile each;
//   * warp 9, the issuer: one thread issues S_X = Q_X . K^T (128 x 128 x D) and
//     O_X += P_X . V (128 x D x 128) for X = A, B;
//   * warps 0-3 and 4-7, the softmax warps of A and B: thread r owns row r
//     (tensor-memory lane r): running max and sum in registers, weights P back
//     into tensor memory as 16-bit pairs over the columns of S, O rescaled there
//     when the max has grown by more than 2^8.  A weight may be above 1 until
//     then (16-bit weights round relatively, so none is the worse for it); one
//     that would pass 2^24 (fp16: 2^15) moves the maximum at once.
// While the softmax warps of one block work, the tensor core runs the other
// block's products.  Tensor memory: S_A, S_B of 128 columns (P_X over the first
// 64 of S_X), O_A, O_B of D columns: all 512 for D = 128.
//
// A value row whose key no row sees must be zeros (a zero weight times a stale
// NaN is NaN).  A prefix's tensor maps end where it ends (its last page has a
// map of its own), and TMA fills what lies outside a map with zeros; a
// sequence's end and bounds are known on the device only, and A's softmax warps
// zero such rows before they hand over their weights (the issuer waits for A's
// weights before either block's P . V).
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

constexpr int kCols = 64;  // columns of S that a softmax thread takes at a time

// kSlots: ring slots (a K or a V tile each).
template <int D, int kSlots_> struct PairTc5Shape {
    static constexpr int kTK = 128;
    static constexpr int kBoxes = D / 64;               // 128-byte column boxes of a row
    static constexpr int kBoxBytes = kTK * 128;         // one column box of a tile (or Q block)
    static constexpr int kTileBytes = kBoxes * kBoxBytes;
    static constexpr int kSlots = kSlots_;
    static constexpr int kThreads = 320;
    static constexpr int kTmemCols = 512;
    static constexpr int kTmemS = 0, kTmemO = 256;      // S_X at 128 X; O_X at 256 + D X
    static constexpr int kQOff = kSlots * kTileBytes;
    static constexpr int kBarOff = kQOff + 2 * kTileBytes;
    // full[kSlots], empty[kSlots], q_full, q_empty, s_full[2], p_full[2], pv_done[2], mma_done
    static constexpr int kNumBars = 2 * kSlots + 9;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // tensor-memory base, abort flag
    static constexpr int kSmemBytes = kMiscOff + 16;         // (the job's tables follow)
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
__device__ __forceinline__ bool pair_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort)
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

// A pair of weights times a factor.
template <typename T> __device__ __forceinline__ uint32_t scale_pair(uint32_t w, float f)
{
    float lo, hi;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xffff0000u);
    } else {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        lo = v.x;
        hi = v.y;
    }
    return pack_pair<T>(lo * f, hi * f);
}

// tcgen05.ld of 16 consecutive 32-bit columns of this thread's lane, waited for.
__device__ __forceinline__ void tc5_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// tcgen05.ld of 64 consecutive 32-bit columns of this thread's lane, waited for.
__device__ __forceinline__ void tc5_ld(uint32_t taddr, uint32_t (&r)[64])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc5_ld(uint32_t taddr, uint32_t (&r)[32]) { tc5_ld32(taddr, r); }

// tcgen05.st of 16 consecutive 32-bit columns of this thread's lane; not waited
// for (tc5_st_wait).
__device__ __forceinline__ void tc5_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc5_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        :
        : "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
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

// One half's place in its tensor map: row y of head z of page (or sequence) w.
struct KeyBox {
    int row, head, page;
    bool last_map;  // values: the map of the prefix's last page
};

// ---- a batch's rows over one shared prefix (kvd_prefix.cuh) ----
template <typename T, int D, bool kPaged> struct PrefixJob {
    using Args = PrefixArgs;
    static constexpr bool kMod = false;
    static constexpr int kSlots = D == 128 ? 5 : 6;
    const Args &a;
    int t, lo, hi, u, k;

    __device__ static void tables(const Args &, int *, int) {}
    // No griddepcontrol.wait before the work: this kernel's CTAs start once every
    // CTA of the launch before it (the same call's attention over the own
    // caches) has passed its own wait for everything older, and that launch
    // writes nothing that is read or written here.
    static constexpr bool kWaitFirst = false;
    __device__ PrefixJob(const Args &args, const int *) : a(args)
    {
        prefix_range(a, &lo, &hi);
        t = lo;
        u = lo / a.n_tiles;
        k = lo % a.n_tiles;
    }
    __device__ bool more() const { return t < hi; }
    __device__ bool first() const { return t == lo || k == 0; }
    __device__ bool last() const { return t == hi - 1 || k == a.n_tiles - 1; }
    __device__ int blocks_here() const { return min(a.unit_blocks, a.blocks - (u % a.units_per_head) * a.unit_blocks); }
    __device__ void next()
    {
        ++t;
        if (++k == a.n_tiles) {
            k = 0;
            ++u;
        }
    }
    __device__ int key(int half) const { return k * 128 + half * 64; }
    __device__ bool has(int half) const { return key(half) < a.S; }
    __device__ int k_end() const { return a.S; }
    // (a half past the prefix: rows past the map's end, which load as zeros)
    __device__ KeyBox box(int half) const
    {
        KeyBox x{key(half), u / a.units_per_head, 0, !kPaged};
        if constexpr (kPaged) {
            const int last_page = (a.S - 1) >> a.page_shift, lp = min(x.row >> a.page_shift, last_page);
            x.row -= lp << a.page_shift;
            x.last_map = lp == last_page;
            x.page = __ldg(a.table + lp);
        }
        return x;
    }
    // the piece's Q blocks; 4-D boxes gather the sequences' rows
    __device__ void load_q(unsigned char *dst, int tile_bytes, int box_bytes, const CUtensorMap *map, uint64_t *bar) const
    {
        const int nb = blocks_here(), b0 = (u % a.units_per_head) * a.unit_blocks;
        const uint32_t bytes = (uint32_t)(a.row_blocks == 1 ? a.seqs * a.gN : kPrefixBlock) * 128u;
        mbar_arrive_expect_tx(bar, bytes * (uint32_t)(nb * (D / 64)));
        for (int x = 0; x < nb; ++x) {
            const int2 o = prefix_block_origin(a, b0 + x);
#pragma unroll
            for (int bx = 0; bx < D / 64; ++bx)
                tma_load_4d(dst + x * tile_bytes + bx * box_bytes, map, bx * 64, o.y, u / a.units_per_head, o.x, bar);
        }
    }
    __device__ void begin(int, int) {}
    __device__ void tile() {}
    __device__ __forceinline__ void scores(uint32_t (&s)[kCols], int c, bool) const
    {
        const int left = a.S - (k * 128 + c * kCols);
        if (left < kCols) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                if (i >= left) s[i] = 0xff800000u;  // -inf
        }
    }
    __device__ bool maximum_modified() const { return false; }
    __device__ float maximum(float top) const { return top * a.qscale; }
    __device__ float exponent_scale() const { return a.qscale; }
    // Row r of block x: its piece's state, columns c0 .. c0 + 31 of o at a time.
    __device__ void store(int x, int r, int c0, const uint32_t (&o)[32], float m, float l) const
    {
        const size_t slot = (size_t)(u + (int)blockIdx.x);
        const int sr = x * kPrefixBlock + r;
        float4 *po = reinterpret_cast<float4 *>(a.part) + slot * (D / 4) * a.slot_rows + sr;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            __stcg(po + (size_t)((c0 + i) / 4) * a.slot_rows,
                   make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                               __uint_as_float(o[i + 3])));
        if (c0 == 0) {
            a.part_ml[slot * 2 * a.slot_rows + sr] = m;
            a.part_ml[(slot * 2 + 1) * a.slot_rows + sr] = l;
        }
    }
};

// ---- a sequence's rows with modified scores ----
//
// A unit is a pair of row blocks of one (b, h); its tiles are the 64-key tiles
// of the sequence's regions, two by two (a pair may span a gap).  Units and
// tiles form one list in which each unit costs kPieceUnits tiles more than it
// has; CTA c of G takes an equal range.  A CTA holds at most two pieces of units
// that it shares: slot 2 c for the one it continues, 2 c + 1 for the one it
// starts.  AttnScoredArgs: n_rowblocks is the pairs per (b, h), part the slots
// ([D / 4][slot_rows] float4 each, then [2][slot_rows] m and l of all slots),
// merge_state int2 (first CTA, CTAs) per unit.
constexpr int kPairPieceUnits = 2;
__device__ __forceinline__ int pair_slot_rows(const AttnScoredArgs &a) { return a.rows > 128 ? 256 : 128; }
__device__ __forceinline__ float *pair_ml(const AttnScoredArgs &a, int D, int grid)
{
    return a.part + (size_t)2 * grid * pair_slot_rows(a) * D;
}

template <typename T, int D, bool kPaged> struct ScoredJob {
    using Args = AttnScoredArgs;
    static constexpr bool kMod = true;
    static constexpr int kSlots = D == 128 ? 4 : 6;  // (the sequences' tables take the fifth's place)
    static constexpr bool kWaitFirst = true;
    const Args &a;
    const int *pre, *pl;
    long long t, hi, n, G;
    int b, hr, k, nt, HR;
    bool start;
    TileRegions reg;  // of 64-key tiles
    // softmax warps: the row's bounds, its sequence's
    RowScore rs;
    ModTile mod;
    int key0, key1;
    bool open;

    // One warp: pre[b] = cost of sequences 0 .. b-1 per unit, pl[b] = P_b, then
    // the sequences' first document keys and prefix lengths.
    __device__ static void tables(const Args &a, int *pre, int lane)
    {
        int *pl = pre + a.B + 1;
        int carry = 0;
        if (lane == 0) pre[0] = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            int units = 0;
            if (b < a.B) {
                const int P = __ldg(a.past_len + b);
                const bool ok = past_len_ok(P, a.N, a.T_max, a.max_past_len);
                if (!ok && blockIdx.x == 0) raise_error(a.err_word, KVD_DEVERR_PAST_LEN);
                if (ok) {
                    const int2 db = seq_bounds(a, b, P);
                    units = (tile_regions<64>(P, a.N, a.window, db.x, db.y).n_tiles + 1) / 2 + kPairPieceUnits;
                    pl[a.B + b] = db.x;
                    pl[2 * a.B + b] = db.y;
                }
                pl[b] = P;
            }
            int v = units;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int m = __shfl_up_sync(0xffffffffu, v, off);
                if (lane >= off) v += m;
            }
            if (b < a.B) pre[b + 1] = carry + v;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __device__ ScoredJob(const Args &args, const int *tables) : a(args), pre(tables), pl(tables + args.B + 1)
    {
        HR = a.H_kv * a.n_rowblocks;
        n = (long long)pre[a.B] * HR;
        G = min((long long)gridDim.x, n);
        t = hi = 0;
        start = true;
        if (blockIdx.x >= G) return;
        const long long lo = n * blockIdx.x / G;
        hi = n * (blockIdx.x + 1) / G;
        int b_lo = 0, b_hi = a.B - 1;  // last b with pre[b] * HR <= lo
        while (b_lo < b_hi) {
            const int mid = (b_lo + b_hi + 1) / 2;
            if ((long long)pre[mid] * HR <= lo) b_lo = mid; else b_hi = mid - 1;
        }
        b = b_lo;
        const int cost = pre[b + 1] - pre[b];
        nt = cost - kPairPieceUnits;
        const long long local = lo - (long long)pre[b] * HR;
        hr = (int)(local / cost);
        k = max(0, (int)(local % cost) - kPairPieceUnits);
        t = (long long)pre[b] * HR + (long long)hr * cost + kPairPieceUnits + k;
        if (t < hi) enter();
    }
    __device__ void enter() { reg = tile_regions<64>(pl[b], a.N, a.window, pl[a.B + b], pl[2 * a.B + b]); }
    __device__ bool more() const { return t < hi; }
    __device__ bool first() const { return start; }
    __device__ bool last() const { return k == nt - 1 || t == hi - 1; }
    __device__ int pair() const { return hr % a.n_rowblocks; }
    __device__ int blocks_here() const { return a.rows > pair() * 256 + 128 ? 2 : 1; }
    __device__ void next()
    {
        ++t;
        start = false;
        if (++k == nt) {
            k = 0;
            start = true;
            if (++hr == HR) {
                hr = 0;
                do {
                    ++b;
                } while (b < a.B && pre[b + 1] == pre[b]);
                if (b < a.B) nt = pre[b + 1] - pre[b] - kPairPieceUnits;
            }
            t += kPairPieceUnits;
            if (t < hi) enter();
        }
    }
    __device__ bool has(int half) const { return 2 * k + half < reg.n_tiles; }
    __device__ int key(int half) const { return reg.tile(has(half) ? 2 * k + half : 2 * k) * 64; }
    __device__ int k_end() const { return pl[b] + a.N; }
    __device__ KeyBox box(int half) const
    {
        KeyBox x{key(half), hr / a.n_rowblocks, b, false};
        if constexpr (kPaged) {
            x.page = __ldg(a.block_table + (size_t)b * (a.T_max >> a.page_shift) + (x.row >> a.page_shift));
            x.row &= (1 << a.page_shift) - 1;
        }
        return x;
    }
    __device__ void load_q(unsigned char *dst, int tile_bytes, int box_bytes, const CUtensorMap *map, uint64_t *bar) const
    {
        const int nb = blocks_here();
        const int row = (b * a.H_kv + hr / a.n_rowblocks) * a.rows + pair() * 256;
        mbar_arrive_expect_tx(bar, (uint32_t)(nb * tile_bytes));  // (rows past the head's: the next head's, not used)
        for (int x = 0; x < nb; ++x)
#pragma unroll
            for (int bx = 0; bx < D / 64; ++bx)
                tma_load_4d(dst + x * tile_bytes + bx * box_bytes, map, bx * 64, row + x * 128, 0, 0, bar);
    }
    // A piece starts, for row r of block x.
    __device__ void begin(int x, int r)
    {
        const int P = pl[b];
        mod = mod_tile(a, nullptr, b, P);
        rs = row_score(a, b, hr / a.n_rowblocks, pair() * 256 + x * 128 + r, P);
        if (x == 0 && r == 0 && k == 0) {  // how the unit is split, for the join
            const int c0 = owner_cta(t, n, G);
            static_cast<int2 *>(a.merge_state)[(size_t)b * HR + hr] = make_int2(c0, owner_cta(t + nt - 1, n, G) - c0 + 1);
        }
    }
    __device__ void store(int x, int r, int c0, const uint32_t (&o)[32], float m, float l) const
    {
        const int rg = pair() * 256 + x * 128 + r;
        if (rg >= a.rows) return;
        const int bh = b * a.H_kv + hr / a.n_rowblocks;
        const int cf = owner_cta(t - k, n, G);
        if (owner_cta(t - k + nt - 1, n, G) == cf) {  // the whole unit lies here
            if (a.row_state != nullptr) {
                float *pr = a.row_state + ((size_t)bh * a.rows + rg) * (D + 4);
#pragma unroll
                for (int i = 0; i < 32; i += 4) *reinterpret_cast<uint4 *>(pr + c0 + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                if (c0 == 0) *reinterpret_cast<float2 *>(pr + D) = make_float2(m, l);
                return;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;  // (a row that sees nothing: zeros)
            T *row = static_cast<T *>(a.out) + ((size_t)bh * a.rows + rg) * D + c0;
#pragma unroll
            for (int i = 0; i < 32; i += 8)
                stg128(row + i, make_uint4(pack_pair<T>(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv),
                                           pack_pair<T>(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv),
                                           pack_pair<T>(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv),
                                           pack_pair<T>(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv)));
            return;
        }
        const size_t slot = (size_t)blockIdx.x * 2 + ((int)blockIdx.x == cf ? 1 : 0);
        const int rows = pair_slot_rows(a), sr = x * 128 + r;
        float4 *po = reinterpret_cast<float4 *>(a.part) + slot * (D / 4) * rows + sr;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            __stcg(po + (size_t)((c0 + i) / 4) * rows,
                   make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                               __uint_as_float(o[i + 3])));
        if (c0 == 0) {
            float *ml = pair_ml(a, D, (int)gridDim.x) + slot * 2 * rows + sr;
            ml[0] = m;
            ml[rows] = l;
        }
    }
    // A tile starts: its halves' keys, and whether the row sees all of them.
    __device__ void tile()
    {
        key0 = key(0);
        key1 = key(1);
        open = has(1) && max(key0, key1) + 64 <= k_end() && row_sees_all<64>(rs, mod.pre, key0) &&
               row_sees_all<64>(rs, mod.pre, key1);
    }
    // The c-th kCols columns of the tile's raw scores, bounded (-inf), and
    // with `modify` modified first (to log2 units; a cap alone keeps the order of
    // scores, so a row's maximum is capped rather than its scores).
    __device__ __forceinline__ void scores(uint32_t (&s)[kCols], int c, bool modify) const
    {
        const int half = c * kCols / 64, base = (half == 0 ? key0 : key1) + c * kCols % 64;
        if (modify) {
            if (a.cap > 0.f) {
                const float in = a.qscale * a.cap_in;
                const f32x2 in2 = pack2(in, in), one2 = pack2(1.f, 1.f);
                // (cap_score for two with one reciprocal (one each: 84 us for the
                // capped chunk's 77): 1 / a and 1 / b from
                // 1 / (a b), the exponents limited to 2^60, where tanh is 1)
#pragma unroll
                for (int i = 0; i < kCols; i += 2) {
                    float x0, x1;
                    unpack2(mul2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), in2), x0, x1);
                    const f32x2 e = add2(pack2(fast_exp2(fminf(x0, 60.f)), fast_exp2(fminf(x1, 60.f))), one2);
                    float e0, e1, r;
                    unpack2(e, e0, e1);
                    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e0 * e1));
                    r *= -2.f * a.cap;
                    s[i] = __float_as_uint(fmaf(r, e1, a.cap));
                    s[i + 1] = __float_as_uint(fmaf(r, e0, a.cap));
                }
            }
            if (a.slopes != nullptr) {
                const float d0 = (float)(rs.p - base), q = a.cap > 0.f ? 1.f : a.qscale;
#pragma unroll
                for (int i = 0; i < kCols; ++i)  // (whole numbers: d0 - i is exact below 2^24)
                    s[i] = __float_as_uint(fmaf(-rs.slope, fabsf(d0 - (float)i), __uint_as_float(s[i]) * q));
            }
        }
        if (!open) {
            const int end = has(half) ? k_end() : base;
#pragma unroll
            for (int i = 0; i < kCols; ++i)
                if (base + i >= end || !row_sees(rs, mod.pre, base + i)) s[i] = 0xff800000u;
        }
    }
    // Whether a maximum has to be taken over modified scores; a raw maximum in
    // log2 units; what the exponents multiply the scores by.
    __device__ bool maximum_modified() const { return a.slopes != nullptr; }
    __device__ float maximum(float top) const
    {
        if (a.slopes != nullptr || top == __int_as_float(0xff800000)) return top;
        return a.cap > 0.f ? cap_score<false>(top * a.qscale, a.cap, a.cap_in) : top * a.qscale;
    }
    // Whether value row r of the tile must be zeroed.
    __device__ bool some_zero() const
    {
        return !has(1) || some_unseen(mod, key(0), 64, k_end()) || some_unseen(mod, key(1), 64, k_end());
    }
    __device__ bool zero_row(int r) const
    {
        const int half = r / 64;
        return !has(half) || key_unseen(mod, key(half) + r % 64, k_end());
    }
    __device__ float exponent_scale() const { return a.cap > 0.f || a.slopes != nullptr ? 1.f : a.qscale; }
};

// Join of the units that several CTAs share: 32 rows of a block and 32 columns
// per CTA, as prefix_join_kernel.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) pair_join_kernel(const AttnScoredArgs a, const int grid, const int blocks)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int chunk = blockIdx.x % 4, k = blockIdx.x / 4 % blocks, bh = blockIdx.x / 4 / blocks;
    const int rg = k * 128 + chunk * 32 + lane, c0 = blockIdx.y * (kJoinThreads / 32) + warp;
    const int b = bh / a.H_kv;
    const int P = __ldg(a.past_len + b);
    const int2 seg = __ldcg(static_cast<const int2 *>(a.merge_state) + (size_t)bh * a.n_rowblocks + k / 2);
    if (rg >= a.rows || !past_len_ok(P, a.N, a.T_max, a.max_past_len) || seg.y <= 1) return;
    if (seg.x < 0 || seg.y > grid - seg.x) return;  // (not written: a CTA gave up)
    PieceJoin<D> j;
    const int rows = pair_slot_rows(a), sr = k % 2 * 128 + chunk * 32 + lane;
    const float *ml = pair_ml(a, D, grid);
    j.template pieces<false>(reinterpret_cast<const float4 *>(a.part), ml, rows, sr, c0, seg.y,
             [&](int i) { return (size_t)(seg.x + i) * 2 + (i == 0 ? 1 : 0); });
    j.template write<T>(static_cast<T *>(a.out) + ((size_t)bh * a.rows + rg) * D + c0 * 4);
}

template <typename T, int D, template <typename, int, bool> class JobOf, bool kPaged>
__global__ void __launch_bounds__(320, 1)
    pair_tc5_kernel(const typename JobOf<T, D, kPaged>::Args a, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_v_last,
                    const __grid_constant__ CUtensorMap tm_q)
{
    using Job = JobOf<T, D, kPaged>;
    using S = PairTc5Shape<D, Job::kSlots>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr float kRescaleThreshold = 8.0f;
    constexpr float kLateLimit = kBf16 ? 24.0f : 15.0f;  // (fp16 weights end at 2^16)
    const float kNegInf = __int_as_float(0xff800000);
    extern __shared__ __align__(1024) unsigned char smem_pair[];
    unsigned char *smem = smem_pair;
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
    int *tables = reinterpret_cast<int *>(smem + S::kSmemBytes);
    if constexpr (Job::kWaitFirst) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (warp == 8) Job::tables(a, tables, lane);
    }
    tc5_fence_before();
    __syncthreads();
    tc5_fence_after();
    const uint32_t tmem = misc[0];
    Job job(a, tables);  // (every thread walks the CTA's tiles itself)

    if (warp == 8) {
        // ---- producer ----
        if (lane == 0) {
            int fills = 0, q_loads = 0;
            bool dead = false;
            // the next ring slot, free
            auto take = [&]() -> int {
                const int s = fills % S::kSlots;
                if (fills >= S::kSlots && !pair_wait(&empty[s], (uint32_t)(fills / S::kSlots - 1) & 1u, abort)) return -1;
                ++fills;
                return s;
            };
            auto load_tile = [&](const CUtensorMap *map, const CUtensorMap *map_last, uint32_t extra) -> bool {
                const int s = take();
                if (s < 0) return false;
                unsigned char *dst = smem + s * S::kTileBytes;
                mbar_arrive_expect_tx(&full[s], (uint32_t)S::kTileBytes + extra);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    KeyBox x = job.box(half);
                    if constexpr (kPaged) {
                        if ((unsigned)x.page >= (unsigned)a.num_pages) {  // never read outside the pool
                            raise_error(a.err_word, KVD_DEVERR_PAGE);
                            x.page = 0;
                        }
                    }
                    const CUtensorMap *m = x.last_map ? map_last : map;
#pragma unroll
                    for (int bx = 0; bx < S::kBoxes; ++bx)
                        tma_load_4d(dst + bx * S::kBoxBytes + half * 64 * 128, m, bx * 64, x.row, x.head, x.page, &full[s]);
                }
                return true;
            };
            uint32_t extra = 0u;
#ifdef KVD_TIMEOUT_TEST
            if (a.flags & kArgTestStall) extra = 16u;  // a stage that never completes
#endif
            for (; job.more() && !dead; job.next()) {
                if (job.first()) {  // a piece starts: its Q blocks
                    if (q_loads > 0 && !pair_wait(q_empty, (uint32_t)(q_loads - 1) & 1u, abort)) {
                        dead = true;
                        break;
                    }
                    job.load_q(smem + S::kQOff, S::kTileBytes, S::kBoxBytes, &tm_q, q_full);
                    ++q_loads;
                }
                dead = !load_tile(&tm_k, &tm_k, extra) || !load_tile(&tm_v, &tm_v_last, 0u);
                extra = 0u;
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
            uint32_t pieces = 0u, n0 = 0u, n1 = 0u;  // pieces, and tiles of each block, so far
            bool have_s = false;                     // S of this tile is issued already
            while (job.more()) {
                const bool two = job.blocks_here() > 1;
                const bool first = job.first(), last = job.last();
                job.next();
                const bool next_last = job.more() && job.last();
                if (!have_s) {
                    ok = pair_wait(q_full, pieces & 1u, abort) && pair_wait(&full[slot], par, abort);
                    ++pieces;
                    // (S_X lies over the previous piece's last P_X)
                    if (ok && n0 > 0u) ok = pair_wait(&pv_done[0], (n0 - 1u) & 1u, abort);
                    if (ok && two && n1 > 0u) ok = pair_wait(&pv_done[1], (n1 - 1u) & 1u, abort);
                    if (!ok) break;
                    tc5_fence_after();
                    issue_s(0, slot);
                    if (two) issue_s(1, slot);
                    tc5_commit(&empty[slot]);
                    if (last) tc5_commit(q_empty);
                    step();
                }
                const int vs = slot;
                if (!(ok = pair_wait(&full[vs], par, abort) && pair_wait(&p_full[0], n0 & 1u, abort))) break;
                step();
                const int ks = slot;  // the next tile's K
                tc5_fence_after();
                issue_pv(0, vs, first);
                if (!two) tc5_commit(&empty[vs]);
                if (!last) {  // the next tile's S of this block, once its P . V is complete
                    if (!(ok = pair_wait(&full[ks], par, abort) && pair_wait(&pv_done[0], n0 & 1u, abort))) break;
                    issue_s(0, ks);
                    if (!two) tc5_commit(&empty[ks]);
                }
                ++n0;
                if (two) {
                    if (!(ok = pair_wait(&p_full[1], n1 & 1u, abort))) break;
                    tc5_fence_after();
                    issue_pv(1, vs, first);
                    tc5_commit(&empty[vs]);
                    if (!last) {
                        if (!(ok = pair_wait(&pv_done[1], n1 & 1u, abort))) break;
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
        // m_run: what the exponents subtract; m_seen: the row's true maximum so far
        float m_run = kNegInf, m_seen = kNegInf, l_run = 0.f;
        uint32_t n_s = 0u;
        bool dead = false;
        auto warp_wait = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, pair_wait(bar, parity & 1u, abort));
        };
        for (int it = 0; job.more(); job.next(), ++it) {  // it: tiles of the CTA so far
            const bool first = job.first(), last = job.last();
            if (x < job.blocks_here()) {
                if (first) {
                    job.begin(x, r);
                    m_run = m_seen = kNegInf;
                    l_run = 0.f;
                }
                job.tile();
                if (!warp_wait(&s_full[x], n_s)) {
                    dead = true;
                    break;
                }
                tc5_fence_after();
                // O, the sum and the maximum move to a larger maximum (rows that
                // keep theirs: by a factor of 1).
                auto raise = [&](bool grows, float to) {
                    if (!__any_sync(0xffffffffu, grows)) return;
                    const float alpha = grows ? fast_exp2(m_run - to) : 1.f;
                    if (grows) m_run = to;
                    l_run *= alpha;
                    if (first) return;  // (no O yet)
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tc5_ld32(t_o + c0, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tc5_st32(t_o + c0, o);
                    }
                };
                auto chunk_max = [&](const uint32_t (&s)[kCols]) -> float {
                    float m4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                    for (int i = 0; i < kCols; i += 2) m4[(i / 2) & 3] = max3(m4[(i / 2) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                    return max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
                };
                // kCols columns at a time and rolled: over the whole tile, the scores
                // alone are 128 registers, and modified scores' code outgrows the
                // instruction cache (a capped 128-token chunk 118 us unrolled, 91 in
                // steps of 32).  Steps of 64 against 32, which wait twice as often for
                // tensor memory: the chunk 77 / 81 us, a prefix of 16384 keys for 128
                // sequences 69.2 / 73.0.
                // The maximum of a tile is taken with its weights, whose exponents
                // subtract the maximum before it: a pass of its own (taken only while
                // some row of the warp has seen nothing) took 91 us where this takes
                // 81.  Sixteen softmax warps, two threads a row: 80.
                if (__any_sync(0xffffffffu, m_run == kNegInf)) {
                    float mx = kNegInf;
#pragma unroll 1
                    for (int c = 0; c < 128 / kCols; ++c) {
                        uint32_t s[kCols];
                        tc5_ld(t_s + kCols * c, s);
                        job.scores(s, c, job.maximum_modified());
                        mx = fmaxf(mx, chunk_max(s));
                    }
                    m_seen = fmaxf(m_seen, job.maximum(mx));
                }
                raise(m_seen > m_run + kRescaleThreshold, m_seen);
                const float escale = job.exponent_scale();
                float l_tile = 0.f;
#pragma unroll 1
                for (int c = 0; c < 128 / kCols; ++c) {  // (weights over columns that are read)
                    uint32_t s[kCols], pk[kCols / 2];
                    tc5_ld(t_s + kCols * c, s);
                    job.scores(s, c, true);
                    const float top = chunk_max(s) * escale;
                    m_seen = fmaxf(m_seen, top);
                    if (const bool late = top > m_run + kLateLimit; __any_sync(0xffffffffu, late)) {
                        // by a power of two: the weights that are written scale exactly
                        const float to = late ? m_run + floorf(top - m_run) : m_run;
                        const float alpha = late ? fast_exp2(m_run - to) : 1.f;
                        l_tile *= alpha;
                        tc5_st_wait();
                        for (int w = 0; w < c * kCols / 32; ++w) {
                            uint32_t pw[16];
                            tc5_ld16(t_s + 16 * w, pw);
#pragma unroll
                            for (int i = 0; i < 16; ++i) pw[i] = scale_pair<T>(pw[i], alpha);
                            tc5_st16(t_s + 16 * w, pw);
                        }
                        raise(late, to);
                    }
                    // weights 2^(escale s - m): scale and maximum in one packed FMA,
                    // sums as packed pairs in two chains
                    const float nmu = (m_run == kNegInf) ? 0.f : -m_run;
                    const f32x2 q2 = pack2(escale, escale), nmu2 = pack2(nmu, nmu);
                    f32x2 l2[2] = {0ull, 0ull};
#pragma unroll
                    for (int i = 0; i < kCols / 2; ++i) {
                        float y0, y1;
                        unpack2(fma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), q2, nmu2), y0, y1);
                        const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
                        l2[i & 1] = add2(l2[i & 1], pack2(p0, p1));
                        pk[i] = pack_pair<T>(p0, p1);
                    }
#pragma unroll
                    for (int w = 0; w < kCols / 2; w += 16) tc5_st16(t_s + c * (kCols / 2) + w, pk + w);
                    float le, lo2;
                    unpack2(add2(l2[0], l2[1]), le, lo2);
                    l_tile += le + lo2;
                }
                tc5_st_wait();
                l_run += l_tile;
                if constexpr (Job::kMod) {
                    if (x == 0 && job.some_zero()) {
                        const int fv = 2 * it + 1;  // the tile's V among the ring's fills
                        if (!warp_wait(&full[fv % S::kSlots], (uint32_t)(fv / S::kSlots))) {
                            dead = true;
                            break;
                        }
                        if (job.zero_row(r)) {
                            const uint32_t vt = smem_addr(smem + (fv % S::kSlots) * S::kTileBytes);
#pragma unroll
                            for (int c = 0; c < D / 8; ++c) {
                                const uint32_t lin = vt + (c >> 3) * S::kBoxBytes + r * 128 + ((c & 7) << 4);
                                sts128(lin ^ ((lin >> 3) & 0x70u), make_uint4(0u, 0u, 0u, 0u));
                            }
                        }
                        fence_proxy_async_shared();
                    }
                }
                tc5_fence_before();
                mbar_arrive(&p_full[x]);
                if (last) {
                    // ---- end of a piece: its (o, m, l) ----
                    if (!warp_wait(&pv_done[x], n_s)) {
                        dead = true;
                        break;
                    }
                    tc5_fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tc5_ld32(t_o + c0, o);
                        job.store(x, r, c0, o, m_run, l_run);
                    }
                    tc5_fence_before();  // (the next arrive on p_full orders these reads before O is overwritten)
                }
                ++n_s;
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
    if constexpr (!Job::kWaitFirst) {
        // This grid completes only after the launch before it has: the join,
        // which waits for this grid, may read what both wrote.
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
}

template <typename T> bool pick_pair_prefix(int D, bool paged, PrefixVariant *v)
{
    if (D != 64 && D != 128) return false;
    if (D == 64) {
        v->fn = paged ? reinterpret_cast<const void *>(&pair_tc5_kernel<T, 64, PrefixJob, true>)
                      : reinterpret_cast<const void *>(&pair_tc5_kernel<T, 64, PrefixJob, false>);
        v->join_fn = reinterpret_cast<const void *>(&prefix_join_kernel<T, 64>);
        v->smem_bytes = PairTc5Shape<64, PrefixJob<T, 64, false>::kSlots>::kSmemBytes;
    } else {
        v->fn = paged ? reinterpret_cast<const void *>(&pair_tc5_kernel<T, 128, PrefixJob, true>)
                      : reinterpret_cast<const void *>(&pair_tc5_kernel<T, 128, PrefixJob, false>);
        v->join_fn = reinterpret_cast<const void *>(&prefix_join_kernel<T, 128>);
        v->smem_bytes = PairTc5Shape<128, PrefixJob<T, 128, false>::kSlots>::kSmemBytes;
    }
    v->threads = 320;
    v->tile_keys = 128;
    v->join_grid_y = D / 4 / (kJoinThreads / 32);
    v->tma = true;
    return true;
}

template <typename T> bool pick_pair_scored(int D, bool paged, PairVariant *v)
{
    if (D != 64 && D != 128) return false;
    if (D == 64) {
        v->fn = paged ? reinterpret_cast<const void *>(&pair_tc5_kernel<T, 64, ScoredJob, true>)
                      : reinterpret_cast<const void *>(&pair_tc5_kernel<T, 64, ScoredJob, false>);
        v->join_fn = reinterpret_cast<const void *>(&pair_join_kernel<T, 64>);
        v->fixed_smem_bytes = PairTc5Shape<64, ScoredJob<T, 64, false>::kSlots>::kSmemBytes;
    } else {
        v->fn = paged ? reinterpret_cast<const void *>(&pair_tc5_kernel<T, 128, ScoredJob, true>)
                      : reinterpret_cast<const void *>(&pair_tc5_kernel<T, 128, ScoredJob, false>);
        v->join_fn = reinterpret_cast<const void *>(&pair_join_kernel<T, 128>);
        v->fixed_smem_bytes = PairTc5Shape<128, ScoredJob<T, 128, false>::kSlots>::kSmemBytes;
    }
    return true;
}

}  // namespace kvd
