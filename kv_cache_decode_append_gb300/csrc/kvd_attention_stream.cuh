// kvd_attention_stream.cuh -- attention with modified scores for at most 16
// query rows per KV head over 16-bit caches, every warp streaming its own keys.
//
// The persistent kernels pay for a ring that four warps share, two CTA barriers
// and a prefix scan per piece, which is little on heads of many tiles and most of
// the time on heads of a few (a window, documents, a short cache behind a shared
// prefix).  Here a CTA of four warps takes an equal share of one head's 64-key
// tiles, its warps whole tiles in turn, and no warp waits for another before the
// final join:
//   * a warp copies its keys and values, 8 KB a step, into a ring of its own
//     (cp.async, kDepth steps): with the next step in registers instead, the
//     long-context step took 105 us where the ring takes 95;
//   * S^T = K Q^T (mma.sync m16n8k16, the 16-wide dimension over keys): lane
//     (g, t) reads 16 bytes of keys g and g + 8 at columns 32 j + 8 t, whose four
//     words are the A fragments of two k-steps under a permutation of the
//     contraction index that Q's B fragments share (the same 16 bytes of row g);
//   * O^T += V^T P^T: lane (g, t) reads 16 bytes of keys 2t, 2t+1, 2t+8, 2t+9 at
//     columns 8 g; byte permutes pair the keys, and word i of the chunk is the
//     tile of output columns 8 g + 2 i (rows 0..7) and 8 g + 2 i + 1 (8..15);
//     both reads are free of bank conflicts, the 16-byte chunk c of row r lying
//     at c ^ 4 (r & 1) for K and c ^ (r & 6) for V;
//   * the weights of 16 keys go from S^T's accumulators to B fragments by
//     movmatrix;
//   * a row's maximum is raised only when some score exceeds it by 2^8 (one vote
//     per 16 keys; o / l does not depend on it), so the common step has no
//     shuffles.
// Split: gridDim.y CTAs per head, each the same number of the head's tiles; a
// head of several CTAs leaves their states (o, m, l) in the workspace, and the
// CTA that counts last joins them (or, leaving row states for a later join,
// nobody does).
#pragma once

#include "kvd_attention.cuh"

namespace kvd {

struct StreamArgs {
    int max_splits;  // gridDim.y: slots per head
    int cta_tiles;   // tiles that a CTA takes at most
    int states;      // 1: leave states, no output
};

// How many CTAs share a head of n_tiles tiles (max_splits of them cover the
// longest head); CTA y of n takes tiles [n_tiles y / n, n_tiles (y + 1) / n).
__device__ __forceinline__ int stream_splits(int n_tiles, int cta_tiles, int max_splits)
{
    return min(max_splits, (n_tiles + cta_tiles - 1) / cta_tiles);
}

// 16 bytes global -> shared (a shared-space address), asynchronously; zeros
// when !real (src is not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }
__device__ __forceinline__ uint4 lds128_addr(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

template <int D, int NR> struct StreamShape {
    static constexpr int kThreads = 128;
    static constexpr int kTK = 64;                     // keys per tile
    static constexpr int kStep = D == 128 ? 16 : 32;   // keys per ring step: 4 KB of K and of V
    static constexpr int kRows = 8 * NR;               // query rows of a head, at most
    static constexpr int kRowBytes = D * 2;
    static constexpr int kHalf = kStep * kRowBytes;    // K's (and V's) bytes of a step
    // CTAs per SM that registers allow without spills (16 rows of D = 128: 240
    // registers), and steps in a warp's ring.  Measured with 2 steps and 3 CTAs
    // against 3 steps and 2: the long-context step 95.3 / 96.7 us, a 1024-key
    // window 32.4 / 32.6, 16 x 12 heads of 16 rows over documents 28.2 / 31.2;
    // 16 rows of D = 128 at 2 CTAs with 2 steps / 3: 17.1 / 17.9 us (53 MB).
    // Smaller steps of D = 64 (16 keys, 3 of them) at 4 CTAs: the documents 30.6.
    static constexpr int kCtas = D == 128 && NR == 2 ? 2 : 3;
    static constexpr int kDepth = 2;
    static constexpr int kRingBytes = kDepth * 2 * kHalf;
    static constexpr int kPad = 4;                     // floats of padding per row in the join (bank conflicts)
    static constexpr int kJoinBytes = 4 * kRows * (D + kPad) * 4;  // (over the rings)
    static constexpr int kMlOff = 4 * kRingBytes > kJoinBytes ? 4 * kRingBytes : kJoinBytes;  // m, l of 4 warps; a flag
    static constexpr int kSmemBytes = kMlOff + 2 * 4 * kRows * 4 + 16;
};

// NR: tiles of 8 query rows.
template <typename T, int D, int NR, bool kPaged>
__global__ void __launch_bounds__(128, StreamShape<D, NR>::kCtas) attn_stream_kernel(const AttnScoredArgs a, const StreamArgs sa)
{
    using S = StreamShape<D, NR>;
    using Tq = Elem<T>;
    constexpr int kKb = D / 32;  // 32-column blocks of a key (16 bytes per lane each)
    constexpr int kVb = D / 64;  // 64-column blocks of a value
    constexpr int kRowBytes = S::kRowBytes;
    constexpr float kRescaleThreshold = 8.0f;
    const float kNegInf = __int_as_float(0xff800000);
    extern __shared__ __align__(128) unsigned char smem_stream[];
    float (*s_o)[S::kRows][D + S::kPad] = reinterpret_cast<float (*)[S::kRows][D + S::kPad]>(smem_stream);
    float (*s_m)[S::kRows] = reinterpret_cast<float (*)[S::kRows]>(smem_stream + S::kMlOff), (*s_l)[S::kRows] = s_m + 4;
    int &s_last = *reinterpret_cast<int *>(s_l + 4);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane >> 2, t = lane & 3;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int bh = (int)blockIdx.x, b = bh / a.H_kv, h = bh % a.H_kv;
    const int P = __ldg(a.past_len + b);
    if (!past_len_ok(P, a.N, a.T_max, a.max_past_len)) {  // (the whole CTA)
        if (tid == 0 && h == 0 && blockIdx.y == 0) raise_error(a.err_word, KVD_DEVERR_PAST_LEN);
        return;
    }
    const ModTile mod = mod_tile(a, nullptr, b, P);
    const TileRegions reg = tile_regions<S::kTK>(P, a.N, a.window, mod.doc, mod.pre);
    const int n_splits = stream_splits(reg.n_tiles, sa.cta_tiles, sa.max_splits);
    const int y = (int)blockIdx.y;
    if (y >= n_splits) return;
    const int t_lo = (int)((long long)reg.n_tiles * y / n_splits), t_hi = (int)((long long)reg.n_tiles * (y + 1) / n_splits);
    const int k_end = P + a.N;

    // Q's B fragments (rows past the head's are zero)
    uint4 q[NR][kKb];
    const unsigned char *qg = static_cast<const unsigned char *>(a.q) + (size_t)bh * a.rows * kRowBytes;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int j = 0; j < kKb; ++j) {
            const int row = 8 * n + g;
            q[n][j] = row < a.rows ? ldg128_nc(qg + (size_t)row * kRowBytes + j * 64 + t * 16) : make_uint4(0u, 0u, 0u, 0u);
        }
    RowScore rs[NR][2];
    RowScore every{0x7fffffff, 0, 0, 0.f};  // bounds that hold for every row
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            rs[n][e] = row_score(a, b, h, 8 * n + 2 * t + e, P);
            every.p = min(every.p, rs[n][e].p);
            every.lo = max(every.lo, rs[n][e].lo);
            every.doc = max(every.doc, rs[n][e].doc);
        }
#pragma unroll
    for (int off = 1; off <= 2; off *= 2) {
        every.p = min(every.p, __shfl_xor_sync(0xffffffffu, every.p, off));
        every.lo = max(every.lo, __shfl_xor_sync(0xffffffffu, every.lo, off));
        every.doc = max(every.doc, __shfl_xor_sync(0xffffffffu, every.doc, off));
    }

    // Rows of the tile that holds a step's keys: tile k's first cache row.
    const unsigned char *kg = static_cast<const unsigned char *>(a.k_cache), *vg = static_cast<const unsigned char *>(a.v_cache);
    auto page_of = [&](int tile) -> int {
        if constexpr (kPaged) return __ldg(a.block_table + (size_t)b * (a.T_max >> a.page_shift) + ((tile * S::kTK) >> a.page_shift));
        else return 0;
    };
    auto first_row = [&](int tile, int page) -> long long {
        if constexpr (kPaged) {
            if ((unsigned)page >= (unsigned)a.num_pages) {  // never read outside the pool
                if (lane == 0) raise_error(a.err_word, KVD_DEVERR_PAGE);
                page = 0;
            }
            return (((long long)page * a.H_kv + h) << a.page_shift) + ((tile * S::kTK) & ((1 << a.page_shift) - 1));
        } else {
            return (long long)bh * a.T_max + tile * S::kTK;
        }
    };
    const uint32_t ring = smem_addr(smem_stream) + warp * S::kRingBytes;
    // one step's rows into ring step `st` (rows past the sequence's end: zeros)
    auto copy_step = [&](int st, long long row, int in_tile, int n_keys) {
        // (the rows are contiguous: chunk 32 i + lane; row r0 + i kRowsPer, whose
        // swizzles are c ^ 4 (r & 1) and c ^ (r & 6))
        constexpr int kRowsPer = 512 / kRowBytes;
        const uint32_t kd = ring + st * 2 * S::kHalf, vd = kd + S::kHalf;
        const int r0 = lane / (D / 8), c = lane % (D / 8);
        const size_t src = (size_t)(row + in_tile) * kRowBytes + lane * 16;
        const unsigned char *ks = kg + src, *vs = vg + src;
        const int left = n_keys - in_tile - r0;  // rows of this lane's kind that exist
#pragma unroll
        for (int i = 0; i < S::kHalf / 512; ++i) {
            const int r = r0 + i * kRowsPer;
            const bool real = i * kRowsPer < left;
            cp_async16(kd + i * 512 + r0 * kRowBytes + ((c ^ ((r & 1) << 2)) << 4), ks + i * 512, real);
            cp_async16(vd + i * 512 + r0 * kRowBytes + ((c ^ (r & 6)) << 4), vs + i * 512, real);
        }
    };

    float o[NR][D / 16][4], l[NR][2];
    float m[NR][2], mu[NR][2];  // running maximum; what is subtracted (0 while nothing is seen)
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[n][e] = kNegInf;
            mu[n][e] = 0.f;
            l[n][e] = 0.f;
        }
    }

    // The warp's tiles t_lo + warp, + 4, ...: the copies' place (ti, sub), and
    // behind it the one being computed (tc, subc).
    int ti = t_lo + warp, sub = 0, n_keys = 0, page_next = 0;
    long long row = 0;
    auto enter = [&](int page) {
        const int tile = reg.tile(ti);
        n_keys = min(S::kTK, k_end - tile * S::kTK);
        row = first_row(tile, page);
        if (ti + 4 < t_hi) page_next = page_of(reg.tile(ti + 4));
    };
    if (ti < t_hi) enter(page_of(reg.tile(ti)));
    auto copy_next = [&](int st) {  // (always one group, so that the count of groups tells the step)
        if (ti < t_hi) {
            copy_step(st, row, sub * S::kStep, n_keys);
            if (++sub * S::kStep >= n_keys) {
                sub = 0;
                ti += 4;
                if (ti < t_hi) enter(page_next);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < S::kDepth - 1; ++st) copy_next(st);

    int st = 0, st_copy = S::kDepth - 1;
    for (int tc = t_lo + warp, subc = 0; tc < t_hi;) {
        copy_next(st_copy);
        if (++st_copy == S::kDepth) st_copy = 0;
        cp_async_wait<S::kDepth - 1>();  // this step's rows (of every lane, after the warp barrier)
        __syncwarp();
        const int tile0 = reg.tile(tc) * S::kTK, keys_here = min(S::kTK, k_end - tile0);
#pragma unroll
        for (int half = 0; half < S::kStep / 16; ++half) {
            const int in_tile = subc * S::kStep + half * 16, key0 = tile0 + in_tile;
            const uint32_t kd = ring + st * 2 * S::kHalf + half * 16 * kRowBytes, vd = kd + S::kHalf;
            uint4 kf[2][kKb];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < kKb; ++j)
                    kf[i][j] = lds128_addr(kd + (g + 8 * i) * kRowBytes + (((4 * j + t) ^ ((g & 1) << 2)) << 4));

            // ---- S^T = K Q^T: even and odd k-steps in two chains ----
            float s[NR][4], s2[NR][4];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
#pragma unroll
            for (int j = 0; j < kKb; ++j) {
                const uint32_t a0[4] = {kf[0][j].x, kf[1][j].x, kf[0][j].y, kf[1][j].y};
                const uint32_t a1[4] = {kf[0][j].z, kf[1][j].z, kf[0][j].w, kf[1][j].w};
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    mma_16816<T>(s[n], a0, q[n][j].x, q[n][j].y);
                    mma_16816<T>(s2[n], a1, q[n][j].z, q[n][j].w);
                }
            }
            // ---- scores (log2 units), bounds ----
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = (s[n][e] + s2[n][e]) * a.qscale;
            if (a.cap > 0.f) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] = cap_score<false>(s[n][e], a.cap, a.cap_in);
            }
            if (a.slopes != nullptr) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {  // (whole numbers: exact below 2^24)
                        const float d = (float)(rs[n][e].p - key0 - g);
                        s[n][e] = fmaf(-rs[n][e].slope, fabsf(d), s[n][e]);
                        s[n][e + 2] = fmaf(-rs[n][e].slope, fabsf(d - 8.f), s[n][e + 2]);
                    }
            }
            const bool masked = in_tile + 16 > keys_here || !row_sees_all<16>(every, mod.pre, key0);  // (warp-uniform)
            if (masked) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + g + 8 * (e >> 1);
                        if (key >= k_end || !row_sees(rs[n][e & 1], mod.pre, key)) s[n][e] = kNegInf;
                    }
            }

            // ---- online softmax per query row 2t + (e & 1) ----
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) grow = grow || s[n][e] > m[n][e & 1] + kRescaleThreshold;
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mt = fmaxf(s[n][e], s[n][e + 2]);
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                        if (mt > m[n][e] + kRescaleThreshold) {
                            const float alpha = fast_exp2(m[n][e] - mt);
                            l[n][e] *= alpha;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                o[n][i][e] *= alpha;
                                o[n][i][e + 2] *= alpha;
                            }
                            m[n][e] = mu[n][e] = mt;
                        }
                    }
            }
            uint32_t pb[NR][2];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = fast_exp2(s[n][e] - mu[n][e & 1]);
                    l[n][e & 1] += s[n][e];
                }
                pb[n][0] = movmatrix_trans(pack_pair<T>(s[n][0], s[n][1]));
                pb[n][1] = movmatrix_trans(pack_pair<T>(s[n][2], s[n][3]));
            }

            uint4 vf[4][kVb];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 2 * t + (i & 1) + 8 * (i >> 1);
#pragma unroll
                for (int c = 0; c < kVb; ++c) vf[i][c] = lds128_addr(vd + r * kRowBytes + (((8 * c + g) ^ (r & 6)) << 4));
            }
            // ---- value rows that no row of the sequence sees: zero ----
            if (masked && some_unseen(mod, key0, 16, k_end)) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (key_unseen(mod, key0 + 2 * t + (i & 1) + 8 * (i >> 1), k_end)) {
#pragma unroll
                        for (int c = 0; c < kVb; ++c) vf[i][c] = make_uint4(0u, 0u, 0u, 0u);
                    }
            }

            // ---- O^T += V^T P^T ----
#pragma unroll
            for (int c = 0; c < kVb; ++c) {
                const uint32_t w[4][4] = {{vf[0][c].x, vf[0][c].y, vf[0][c].z, vf[0][c].w},
                                          {vf[1][c].x, vf[1][c].y, vf[1][c].z, vf[1][c].w},
                                          {vf[2][c].x, vf[2][c].y, vf[2][c].z, vf[2][c].w},
                                          {vf[3][c].x, vf[3][c].y, vf[3][c].z, vf[3][c].w}};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t va[4] = {__byte_perm(w[0][i], w[1][i], 0x5410), __byte_perm(w[0][i], w[1][i], 0x7632),
                                            __byte_perm(w[2][i], w[3][i], 0x5410), __byte_perm(w[2][i], w[3][i], 0x7632)};
#pragma unroll
                    for (int n = 0; n < NR; ++n) mma_16816<T>(o[n][4 * c + i], va, pb[n][0], pb[n][1]);
                }
            }
        }
        __syncwarp();  // (the step is read: the next copy may overwrite it)
        if (++st == S::kDepth) st = 0;
        if (++subc * S::kStep >= keys_here) {
            subc = 0;
            tc += 4;
        }
    }
    cp_async_wait<0>();
    __syncthreads();  // (the join lies over the rings)

    // ---- the four warps' states joined through shared memory ----
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
            l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
            l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
            const int r = 8 * n + 2 * t + e;
            if (g == 0) {
                s_m[warp][r] = m[n][e];
                s_l[warp][r] = l[n][e];
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                *reinterpret_cast<float2 *>(&s_o[warp][r][64 * (i / 4) + 8 * g + 2 * (i % 4)]) = make_float2(o[n][i][e], o[n][i][e + 2]);
        }
    __syncthreads();
    const bool single = n_splits == 1 && !sa.states;
    float *slot = a.part + ((size_t)bh * sa.max_splits + y) * a.rows * (D + 4);
    for (int idx = tid; idx < a.rows * (D / 4); idx += S::kThreads) {
        const int r = idx / (D / 4), d = idx % (D / 4) * 4;
        const float M = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
        float den = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float wt = safe_weight(s_m[w][r], M);
            const float4 v = *reinterpret_cast<const float4 *>(&s_o[w][r][d]);
            num.x = fmaf(wt, v.x, num.x);
            num.y = fmaf(wt, v.y, num.y);
            num.z = fmaf(wt, v.z, num.z);
            num.w = fmaf(wt, v.w, num.w);
            den = fmaf(wt, s_l[w][r], den);
        }
        if (single) {
            *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + ((size_t)bh * a.rows + r) * D + d) =
                make_uint2(pack_pair<T>(quotient<true>(num.x, den), quotient<true>(num.y, den)),
                           pack_pair<T>(quotient<true>(num.z, den), quotient<true>(num.w, den)));
        } else {
            *reinterpret_cast<float4 *>(slot + r * (D + 4) + d) = num;
            if (d == 0) *reinterpret_cast<float2 *>(slot + r * (D + 4) + D) = make_float2(M, den);
        }
    }
    if (n_splits == 1 || sa.states) return;

    // ---- the CTA that counts last joins the head's states ----
    __syncthreads();  // every thread's share of the state is written
    int *tickets = static_cast<int *>(a.merge_state);
    if (tid == 0) {
        s_last = atomic_add_acq_rel_gpu(tickets + bh, 1) == n_splits - 1;
        if (s_last) tickets[bh] = 0;  // the next call starts from zero
    }
    __syncthreads();
    if (!s_last) return;
    const float *part = a.part + (size_t)bh * sa.max_splits * a.rows * (D + 4);
    for (int idx = tid; idx < a.rows * (D / 4); idx += S::kThreads) {
        const int r = idx / (D / 4), d = idx % (D / 4) * 4;
        float M = kNegInf, den = 0.f;
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < n_splits; ++k) {
            const float *pr = part + ((size_t)k * a.rows + r) * (D + 4);
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(pr + D));
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(pr + d));
            const float Mn = fmaxf(M, ml.x);
            const float wa = safe_weight(M, Mn), wb = safe_weight(ml.x, Mn);
            num.x = num.x * wa + v.x * wb;
            num.y = num.y * wa + v.y * wb;
            num.z = num.z * wa + v.z * wb;
            num.w = num.w * wa + v.w * wb;
            den = den * wa + ml.y * wb;
            M = Mn;
        }
        *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + ((size_t)bh * a.rows + r) * D + d) =
            make_uint2(pack_pair<T>(quotient<true>(num.x, den), quotient<true>(num.y, den)),
                       pack_pair<T>(quotient<true>(num.z, den), quotient<true>(num.w, den)));
    }
}

constexpr int stream_smem_bytes(int D, int rows)
{
    return D == 64 ? (rows <= 8 ? StreamShape<64, 1>::kSmemBytes : StreamShape<64, 2>::kSmemBytes)
                   : (rows <= 8 ? StreamShape<128, 1>::kSmemBytes : StreamShape<128, 2>::kSmemBytes);
}

constexpr int stream_ctas_per_sm(int D, int rows) { return D == 128 && rows > 8 ? StreamShape<128, 2>::kCtas : StreamShape<64, 1>::kCtas; }

// The kernel for `rows` query rows per KV head (at most 16).
template <typename T> const void *pick_stream_kernel(int D, int rows, bool paged)
{
    if (D == 64) {
        if (rows <= 8)
            return paged ? reinterpret_cast<const void *>(&attn_stream_kernel<T, 64, 1, true>)
                         : reinterpret_cast<const void *>(&attn_stream_kernel<T, 64, 1, false>);
        return paged ? reinterpret_cast<const void *>(&attn_stream_kernel<T, 64, 2, true>)
                     : reinterpret_cast<const void *>(&attn_stream_kernel<T, 64, 2, false>);
    }
    if (rows <= 8)
        return paged ? reinterpret_cast<const void *>(&attn_stream_kernel<T, 128, 1, true>)
                     : reinterpret_cast<const void *>(&attn_stream_kernel<T, 128, 1, false>);
    return paged ? reinterpret_cast<const void *>(&attn_stream_kernel<T, 128, 2, true>)
                 : reinterpret_cast<const void *>(&attn_stream_kernel<T, 128, 2, false>);
}

// kvd_stream_{bf16,f16}.cu
const void *stream_kernel_bf16(int D, int rows, bool paged);
const void *stream_kernel_f16(int D, int rows, bool paged);

}  // namespace kvd
