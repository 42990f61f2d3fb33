// kvd_prefix.cuh -- attention of a batch over one shared prefix.
//
// Every sequence of the batch attends the same prefix keys 0 .. S-1 before its
// own cache.  Softmax splits over any partition of the keys: with (o, m, l) of a
// part (o = sum 2^(y_j - m) v_j, l = sum 2^(y_j - m), y in log2 units),
//   out = sum_parts 2^(m - M) o / sum_parts 2^(m - M) l,   M = max m,
// so the call is three launches on one stream:
//   1. the attention kernels over the sequences' own caches, which leave each
//      row's state instead of an output (AttnScoredArgs::row_state);
//   2. a prefix kernel over the B g N rows that each KV head has in the whole
//      batch: a GEMM-shaped product that reads the prefix once (this file and
//      kvd_pair_tc5.cuh);
//   3. prefix_join_kernel: the join of a row's prefix pieces and own state.
//
// Rows of the prefix kernels.  A KV head's rows are those of its gN rows in
// every sequence (contiguous in q per sequence).  A block is 128 of them: with
// gN <= 128, seqs = 128 / gN whole sequences (seqs gN rows are used); else 128
// rows of one sequence.  A unit is one KV head with `unit_blocks` (1 or 2)
// blocks.
//
// Split.  The (unit, key tile) pairs form one list, unit by unit; CTA c of G
// takes [n c / G, n (c + 1) / G).  A unit's part in one CTA is a piece.  Along
// the list either the unit or the CTA steps from one piece to the next, so piece
// (u, c) has slot u + c: no slot is shared and there are at most units + G - 1.
#pragma once

#include "kvd_attention_stream.cuh"

namespace kvd {

constexpr int kPrefixBlock = 128;  // rows of a block

struct PrefixArgs {
    const void *q;                // [B, H_kv, gN, D]
    const void *k, *v;            // [H_kv, S_max, D], or the page pool
    const int32_t *table;         // paged: pages of the prefix, else null
    float *part;                  // pieces: [slot][(D / 4)][slot_rows] float4 (o), then ...
    float *part_ml;               // ... [slot][2][slot_rows] (m, l)
    uint32_t *err_word;
    int B, H_kv, gN, S, S_max;
    int seqs;                     // sequences per block (gN <= 128), else 1
    int row_blocks;               // blocks per sequence (gN > 128), else 1
    int blocks;                   // blocks per KV head
    int unit_blocks, units_per_head, n_units;
    int n_tiles;                  // key tiles of the prefix
    int slot_rows;                // unit_blocks * 128
    int page_shift, num_pages;
    float qscale;                 // softmax scale * log2(e)
    int flags;                    // (test builds: kArgTestStall)
};

// First sequence and first of its rows of block k of a KV head.
__device__ __forceinline__ int2 prefix_block_origin(const PrefixArgs &a, int k)
{
    return a.row_blocks == 1 ? make_int2(k * a.seqs, 0)
                             : make_int2(k / a.row_blocks, (k % a.row_blocks) * kPrefixBlock);
}

// Sequence and row within it of row r of a block from `origin` (x < 0: none).
__device__ __forceinline__ int2 prefix_block_row(const PrefixArgs &a, int2 origin, int r)
{
    int2 p = origin;
    if (a.row_blocks == 1) {
        p.x += r / a.gN;
        p.y = r % a.gN;
        if (r >= a.seqs * a.gN || p.x >= a.B) p.x = -1;
    } else {
        p.y += r;
        if (p.y >= a.gN) p.x = -1;
    }
    return p;
}

// This CTA's range of the (unit, tile) list.
__device__ __forceinline__ void prefix_range(const PrefixArgs &a, int *lo, int *hi)
{
    const long long n = (long long)a.n_units * a.n_tiles;
    *lo = (int)(n * blockIdx.x / gridDim.x);
    *hi = (int)(n * (blockIdx.x + 1) / gridDim.x);
}

// What the join needs of the attention kernels' row states.
struct RowStateArgs {
    const float *state;   // [B * H_kv * gN][D + 4]: rows of heads that lay in one CTA
    const float *part;    // pieces of the others, as attn_merge_kernel reads them
    const int2 *seg;      // (first CTA, CTAs) per (b, h, row block)
    const int32_t *past_len;
    int rb, n_rowblocks, prow, T_max, max_past_len, N, grid;  // grid: the prefix kernel's CTAs
    int own_grid;               // the attention kernel's CTAs (a bound on seg)
    int pair_grid;              // > 0: part holds the pair kernel's slots (that many CTAs), rb 256
    int max_splits, cta_tiles;  // max_splits > 0: part holds the streaming kernel's slots [B * H_kv][max_splits][gN][D + 4]
};

// Join: out[b, h, y, :] of 32 rows of a block and 32 columns per CTA: a warp
// takes four columns (the pieces' layout: consecutive lanes are consecutive
// rows), a lane one row.  Bound by the latency of reading the pieces (L2): the
// loads of kJoinBatch pieces are in flight together.
constexpr int kJoinThreads = 256;
constexpr int kJoinBatch = 8;

// Four columns of one row, joined part by part.
template <int D> struct PieceJoin {
    float M = -__builtin_huge_valf(), den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);

    __device__ __forceinline__ void add(float m, float l, const float4 &o)
    {
        const float Mn = fmaxf(M, m);
        const float wa = safe_weight(M, Mn), wb = safe_weight(m, Mn);
        den = den * wa + l * wb;
        acc.x = acc.x * wa + o.x * wb;
        acc.y = acc.y * wa + o.y * wb;
        acc.z = acc.z * wa + o.z * wb;
        acc.w = acc.w * wa + o.w * wb;
        M = Mn;
    }
    // n pieces in slots slot_of(0), ... of [D / 4][rows] float4 and [2][rows]
    // floats (m, l): row sr, column group c0.  kMany: a last batch that is not full
    // reads its last piece again instead of testing for each, which parts the
    // loads: faster where pieces are many (a prefix of 1000 keys for 8 sequences,
    // 8 pieces a row: 9.8 / 10.8 us), slower where they are a few (the capped
    // 128-token chunk: 77.3 / 74.1).
    template <bool kMany, typename F>
    __device__ __forceinline__ void pieces(const float4 *part, const float *ml, int rows, int sr, int c0, int n, F slot_of)
    {
        for (int c = 0; c < n; c += kJoinBatch) {
            float m[kJoinBatch], l[kJoinBatch];
            float4 o[kJoinBatch];
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) {
                if (kMany || c + i < n) {
                    const size_t slot = slot_of(min(c + i, n - 1));
                    m[i] = __ldcg(ml + slot * 2 * rows + sr);
                    l[i] = __ldcg(ml + (slot * 2 + 1) * rows + sr);
                    o[i] = __ldcg(part + (slot * (D / 4) + c0) * rows + sr);
                }
            }
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i)
                if (c + i < n) add(m[i], l[i], o[i]);
        }
    }
    template <typename T> __device__ __forceinline__ void write(T *row) const
    {
        const float inv = den == 0.f ? 0.f : 1.f / den;  // (a row that sees nothing: zeros)
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4 *>(row) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        else
            *reinterpret_cast<uint2 *>(row) =
                make_uint2(pack_pair<T>(acc.x * inv, acc.y * inv), pack_pair<T>(acc.z * inv, acc.w * inv));
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const PrefixArgs a, const RowStateArgs s, void *out)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int chunk = blockIdx.x % (kPrefixBlock / 32);
    const int gb = blockIdx.x / (kPrefixBlock / 32);  // block of all heads
    const int h = gb / a.blocks, k = gb % a.blocks;
    const int u = h * a.units_per_head + k / a.unit_blocks;
    const int r = chunk * 32 + lane;                          // row within the block
    const int sr = (k % a.unit_blocks) * kPrefixBlock + r;    // row within the slot
    const int2 p = prefix_block_row(a, prefix_block_origin(a, k), r);
    if (p.x < 0) return;
    const int c0 = blockIdx.y * (kJoinThreads / 32) + warp;   // column group
    const int bh = p.x * a.H_kv + h;
    const int P = __ldg(s.past_len + p.x);
    const int2 seg = s.max_splits > 0 ? make_int2(0, 0) : __ldcg(s.seg + (size_t)bh * s.n_rowblocks + p.y / s.rb);
    if (!past_len_ok(P, s.N, s.T_max, s.max_past_len)) return;  // reported by the first launch
    if (s.max_splits == 0 && (seg.x < 0 || seg.y > s.own_grid - seg.x)) return;  // (not written: a CTA gave up)

    PieceJoin<D> j;
    // the row's own keys
    if (s.pair_grid > 0 && seg.y > 1) {
        const int rows = a.gN > 128 ? 256 : 128;
        j.template pieces<false>(reinterpret_cast<const float4 *>(s.part), s.part + (size_t)2 * s.pair_grid * rows * D, rows, p.y % 256, c0, seg.y,
                 [&](int i) { return (size_t)(seg.x + i) * 2 + (i == 0 ? 1 : 0); });
    } else {
        const int own = s.max_splits > 0 ? stream_splits((P + s.N + 63) / 64, s.cta_tiles, s.max_splits) : seg.y;
        for (int i = 0; i < own; ++i) {
            const float *pr = s.max_splits > 0 ? s.part + (((size_t)bh * s.max_splits + i) * a.gN + p.y) * (D + 4)
                              : seg.y == 1 ? s.state + ((size_t)bh * a.gN + p.y) * (D + 4)
                                           : s.part + (((size_t)(seg.x + i) * 2 + (i == 0)) * s.prow + p.y % s.rb) * (D + 4);
            const float4 o = __ldcg(reinterpret_cast<const float4 *>(pr) + c0);
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(pr + D));
            j.add(ml.x, ml.y, o);
        }
    }
    // the prefix's pieces: the CTAs that hold the unit's tiles (an empty prefix: none)
    const long long n = (long long)a.n_units * a.n_tiles;
    if (n > 0) {
        const int first = owner_cta((long long)u * a.n_tiles, n, s.grid);
        const int last = owner_cta((long long)(u + 1) * a.n_tiles - 1, n, s.grid);
        j.template pieces<true>(reinterpret_cast<const float4 *>(a.part), a.part_ml, a.slot_rows, sr, c0, last - first + 1,
                 [&](int i) { return (size_t)(u + first + i); });
    }
    j.template write<T>(static_cast<T *>(out) + ((size_t)bh * a.gN + p.y) * D + c0 * 4);
}

// Launch facts of a prefix kernel, for the host.
struct PrefixVariant {
    const void *fn;
    const void *join_fn;
    int threads, smem_bytes, tile_keys, join_grid_y;
    bool tma;  // takes the K, V and q tensor maps
};

// The pair kernel with modified scores (kvd_pair_tc5.cuh).
struct PairVariant {
    const void *fn, *join_fn;
    int fixed_smem_bytes;  // plus 4 B + 1 ints
};
bool pair_variant_bf16(int D, bool paged, PairVariant *v);
bool pair_variant_f16(int D, bool paged, PairVariant *v);

bool prefix_variant_f32(int D, bool paged, PrefixVariant *v);
bool prefix_variant_bf16(int D, bool paged, PrefixVariant *v);
bool prefix_variant_f16(int D, bool paged, PrefixVariant *v);

}  // namespace kvd
