// kvd_prefix_simt.cuh -- the shared-prefix kernel of fp32 caches, on the CUDA
// cores (no tensor-core type keeps fp32's 24 bits).
//
// A CTA of 256 threads takes one 128-row block against key tiles of 64: S = Q K^T
// and O += P V as register-tiled products, thread (ty, tx) of 16 x 16 holding
// rows 8 ty .. 8 ty + 7 by keys tx + 16 j (then columns 4 tx + 64 j), the online
// softmax between them over the 16 lanes that share a row.  Bound by FMAs (and
// the shared-memory reads that feed them: 12 16-byte loads for 128 FMAs of S).
// K of the next tile is copied (cp.async) while P V runs, V while S does.
#pragma once

#include "kvd_prefix.cuh"

namespace kvd {

template <int D> struct PrefixSimtShape {
    static constexpr int kTK = 64;
    static constexpr int kThreads = 256;
    static constexpr int kQStride = D + 4, kKStride = D + 4, kPStride = kTK + 4;  // floats per row (no bank conflicts)
    static constexpr int kQOff = 0;
    static constexpr int kKOff = kQOff + kPrefixBlock * kQStride * 4;
    static constexpr int kVOff = kKOff + kTK * kKStride * 4;
    static constexpr int kPOff = kVOff + kTK * D * 4;
    static constexpr int kSmemBytes = kPOff + kPrefixBlock * kPStride * 4;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

template <int D, bool kPaged>
__global__ void __launch_bounds__(256, 1) prefix_simt_kernel(const PrefixArgs a)
{
    using S = PrefixSimtShape<D>;
    constexpr int kCols = D / 64;  // float4 columns of O per thread
    const float kNegInf = __int_as_float(0xff800000);
    extern __shared__ __align__(128) unsigned char smem_simt[];
    float *qs = reinterpret_cast<float *>(smem_simt + S::kQOff), *ks = reinterpret_cast<float *>(smem_simt + S::kKOff);
    float *vs = reinterpret_cast<float *>(smem_simt + S::kVOff), *ps = reinterpret_cast<float *>(smem_simt + S::kPOff);
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    // (no griddepcontrol.wait yet: as the tcgen05 form, PrefixJob::kWaitFirst)
    int lo, hi;
    prefix_range(a, &lo, &hi);

    // one K or V tile into shared memory, rows past the prefix as zeros
    auto load_tile = [&](const void *cache, float *dst, int stride, int h, int tile) {
        const float *base = static_cast<const float *>(cache);
#pragma unroll
        for (int idx = tid; idx < S::kTK * (D / 4); idx += S::kThreads) {
            const int r = idx / (D / 4), c = idx % (D / 4) * 4;
            const int key = tile * S::kTK + r;
            const bool real = key < a.S;
            size_t row = 0;
            if (real) {
                if constexpr (kPaged) {
                    int page = __ldg(a.table + (key >> a.page_shift));
                    if ((unsigned)page >= (unsigned)a.num_pages) {  // never read outside the pool
                        raise_error(a.err_word, KVD_DEVERR_PAGE);
                        page = 0;
                    }
                    row = (((size_t)page * a.H_kv + h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
                } else {
                    row = (size_t)h * a.S_max + key;
                }
            }
            cp_async16(smem_addr(dst + r * stride + c), base + row * D + c, real);
        }
        cp_async_commit();
    };

    float o[8][kCols][4], m[8], l[8];
    int u = lo / a.n_tiles, k = lo % a.n_tiles;
    for (int t = lo; t < hi; ++t) {
        const int h = u / a.units_per_head;
        const bool first = t == lo || k == 0;
        const bool last = t == hi - 1 || k == a.n_tiles - 1;
        if (first) {
            __syncthreads();  // (the previous piece's readers are done)
            const int2 origin = prefix_block_origin(a, u % a.units_per_head);
            for (int idx = tid; idx < kPrefixBlock * (D / 4); idx += S::kThreads) {
                const int r = idx / (D / 4), c = idx % (D / 4) * 4;
                const int2 p = prefix_block_row(a, origin, r);
                float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p.x >= 0)
                    q = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) +
                                                          (((size_t)p.x * a.H_kv + h) * a.gN + p.y) * D + c);
                *reinterpret_cast<float4 *>(qs + r * S::kQStride + c) =
                    make_float4(q.x * a.qscale, q.y * a.qscale, q.z * a.qscale, q.w * a.qscale);
            }
            load_tile(a.k, ks, S::kKStride, h, k);
            load_tile(a.v, vs, D, h, k);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[i] = kNegInf;
                l[i] = 0.f;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][c][e] = 0.f;
            }
        }
        cp_async_wait<1>();  // K of this tile
        __syncthreads();
        float s[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 q[8], kk[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = *reinterpret_cast<const float4 *>(qs + (8 * ty + i) * S::kQStride + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4 *>(ks + (tx + 16 * j) * S::kKStride + d);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(q[i].x, kk[j].x, s[i][j]);
                    s[i][j] = fmaf(q[i].y, kk[j].y, s[i][j]);
                    s[i][j] = fmaf(q[i].z, kk[j].z, s[i][j]);
                    s[i][j] = fmaf(q[i].w, kk[j].w, s[i][j]);
                }
        }
        __syncthreads();  // every thread is done with K
        if (!last) load_tile(a.k, ks, S::kKStride, h, k + 1);
        else cp_async_commit();  // (an empty group keeps the count)
        const int nk = a.S - k * S::kTK;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (tx + 16 * j >= nk) s[i][j] = kNegInf;
            float mt = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
            for (int off = 8; off >= 1; off /= 2) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
            if (mt > m[i]) {  // (a tile has at least one key: mt is finite)
                const float alpha = fast_exp2(m[i] - mt);
                l[i] *= alpha;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][c][e] *= alpha;
                m[i] = mt;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = fast_exp2(s[i][j] - m[i]);
                l[i] += p;  // (this lane's share)
                ps[(8 * ty + i) * S::kPStride + tx + 16 * j] = p;
            }
        }
        cp_async_wait<1>();  // V of this tile
        __syncthreads();
#pragma unroll 2
        for (int kk = 0; kk < S::kTK; kk += 4) {
            float4 p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = *reinterpret_cast<const float4 *>(ps + (8 * ty + i) * S::kPStride + kk);
#pragma unroll
            for (int kq = 0; kq < 4; ++kq)
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const float4 v = *reinterpret_cast<const float4 *>(vs + (kk + kq) * D + 4 * tx + 64 * c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float w = kq == 0 ? p[i].x : kq == 1 ? p[i].y : kq == 2 ? p[i].z : p[i].w;
                        o[i][c][0] = fmaf(w, v.x, o[i][c][0]);
                        o[i][c][1] = fmaf(w, v.y, o[i][c][1]);
                        o[i][c][2] = fmaf(w, v.z, o[i][c][2]);
                        o[i][c][3] = fmaf(w, v.w, o[i][c][3]);
                    }
                }
        }
        __syncthreads();  // every thread is done with V and P
        if (!last) load_tile(a.v, vs, D, h, k + 1);
        else cp_async_commit();
        if (last) {
            const size_t slot = (size_t)(u + (int)blockIdx.x);
            float4 *po = reinterpret_cast<float4 *>(a.part) + slot * (D / 4) * a.slot_rows;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
#pragma unroll
                for (int off = 8; off >= 1; off /= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
                const int r = 8 * ty + i;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    po[(size_t)(tx + 16 * c) * a.slot_rows + r] = make_float4(o[i][c][0], o[i][c][1], o[i][c][2], o[i][c][3]);
                if (tx == 0) {
                    a.part_ml[slot * 2 * a.slot_rows + r] = m[i];
                    a.part_ml[(slot * 2 + 1) * a.slot_rows + r] = l[i];
                }
            }
        }
        if (++k == a.n_tiles) {
            k = 0;
            ++u;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (as pair_tc5_kernel)
}

template <int D> void make_prefix_simt(bool paged, PrefixVariant *v)
{
    v->fn = paged ? reinterpret_cast<const void *>(&prefix_simt_kernel<D, true>)
                  : reinterpret_cast<const void *>(&prefix_simt_kernel<D, false>);
    v->join_fn = reinterpret_cast<const void *>(&prefix_join_kernel<float, D>);
    v->threads = PrefixSimtShape<D>::kThreads;
    v->smem_bytes = PrefixSimtShape<D>::kSmemBytes;
    v->tile_keys = PrefixSimtShape<D>::kTK;
    v->join_grid_y = D / 4 / (kJoinThreads / 32);
    v->tma = false;
}

}  // namespace kvd
