// kvd_rope.cu -- the append with the position rotation applied on the way:
// q and the new keys of N tokens per sequence are rotated by their positions,
// the rotated keys and the values go to their cache slots (contiguous or paged).
//
// Mathematics, per token at position p and frequency f (angle a = p inv_freq[f]):
//   (x, y) -> (x cos a - y sin a, x sin a + y cos a)
// for the pair (x, y) = elements (f, f + rot/2) of the row, or (2f, 2f + 1);
// elements rot .. D-1 and the value rows are copied bit for bit.
//
// Angles of far positions: p inv_freq as an fp32 product is off by up to
// p 2^-24 radians.  Here inv_freq (fp64) becomes turns per position as a 64-bit
// binary fraction (an integer product with 1 / (2 pi) to 128 bits: off by less
// than 2^-63 turns), and the phase is that fraction times p modulo 2^64:
// whole turns drop out exactly in the integer wrap, whatever the position.
// The remaining phase, within an eighth of a turn of its nearest quadrant,
// goes to sinpif / cospif; the rotation itself is fp32, rounded once to the
// cache's type.
//
// Bound: bytes.  Each element of q, k_new and v_new is read once and written
// once; a block takes one token (or, when there are fewer tokens than SMs, a
// share of one token's rows), computes the token's rot/2 angles once into
// shared memory and rotates all its heads with them, so the transcendental work
// is 1 / (H_q + H_kv) of what a thread per element pair would do.  Each thread
// loads its first two units before the angles are needed.  Measured: 2 sequences
// of 2048 tokens, 32 / 8 heads of 128, bf16 (100 MB moved) 19.7 us, 5.1 TB/s (24.2
// with integer divisions where a unit's row now takes a multiplication: the
// instructions, then the angles' barrier, are what bounds it); one step of 32
// sequences 2.4 us, a launch's latency.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvd_device.cuh"
#include "kvd_host.cuh"

namespace kvd {
namespace {

// One call's rows, in 16-byte chunks: strides (of q, k_new, v_new per
// sequence, head, token) and sizes are chunk counts.
struct RopeArgs {
    const uint4 *q, *k_new, *v_new;
    uint4 *q_out, *k_cache, *v_cache;
    const int32_t *past_len;
    const int32_t *positions;    // [B, N] or null: past_len + i
    const int32_t *block_table;  // paged, else null
    const double *inv_freq;      // [rot / 2]
    uint32_t *err_word;
    long long sq[3], sk[3], sv[3];
    int H_q, H_kv, N, T_max, max_past_len;
    int page_shift, max_pages, num_pages;
    int pos_base;
    int n_freq;       // rot / 2
    int row_chunks;   // chunks per row
    int rot_units;    // rotated units per row: a chunk pair (halves) or one chunk (neighbours)
    int row_units;    // rot_units + copied chunks
    int units;        // units of one token: (H_q + H_kv) row_units + H_kv row_chunks
    int split_units;  // units per block of a token (gridDim.y blocks)
    uint64_t inv_row_units, inv_row_chunks;  // ceil(2^36 / row_units), ceil(2^36 / row_chunks)
};

// n / d with inv = ceil(2^36 / d): exact for n < 2^26 and d <= 1024, as
// n (inv d - 2^36) < 2^36.
__device__ __forceinline__ int quotient_of(int n, uint64_t inv) { return (int)(((uint64_t)(uint32_t)n * inv) >> 36); }
constexpr long long kRopeMaxUnits = 1 << 26;

// Turns per position as a 64-bit binary fraction (whole turns dropped), from
// radians per position: bits s .. s+63 of the 181-bit product of f's mantissa
// with 1 / (2 pi) to 128 bits.  Off by less than 2 units of the last place for
// |f| < 2^60.
__device__ __forceinline__ uint64_t turns_from_radians(double f)
{
    // 1 / (2 pi) = (kHi:kLo) 2^-130, rounded down
    constexpr uint64_t kHi = 0xa2f9836e4e441529ull, kLo = 0xfc2757d1f534ddc0ull;
    const uint64_t bits = (uint64_t)__double_as_longlong(f);
    const int e = (int)((bits >> 52) & 0x7ffu);
    if (e == 0) return 0ull;  // (zero; subnormal frequencies never turn)
    const uint64_t m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;  // |f| = m 2^(e - 1075)
    const uint64_t w0 = m * kLo;
    const uint64_t c = __umul64hi(m, kLo), l = m * kHi;
    const uint64_t w1 = l + c, w2 = __umul64hi(m, kHi) + (w1 < l ? 1ull : 0ull);
    const int s = 1141 - e;  // turns 2^64 = (w2:w1:w0) 2^-s
    uint64_t t = 0ull;
    if (s >= 192) t = 0ull;
    else if (s >= 128) t = w2 >> (s - 128);
    else if (s > 64) t = (w1 >> (s - 64)) | (w2 << (128 - s));
    else if (s == 64) t = w1;
    else if (s > 0) t = (w0 >> s) | (w1 << (64 - s));
    else if (s > -64) t = w0 << -s;
    return (bits >> 63) ? 0ull - t : t;
}

// cos and sin of position * frequency, through the exact phase.
__device__ __forceinline__ float2 rotation_of(uint64_t turns, int64_t pos)
{
    const uint32_t phase = (uint32_t)((turns * (uint64_t)pos) >> 32);
    const uint32_t quadrant = (phase + 0x20000000u) >> 30;
    // half turns within -1/4 .. 1/4 of the quadrant's middle
    const float x = (float)(int32_t)(phase - (quadrant << 30)) * 4.656612873077393e-10f;  // 2^-31
    const float s = sinpif(x), c = cospif(x);
    const bool swap = (quadrant & 1u) != 0u;
    float cs = swap ? s : c, sn = swap ? c : s;
    if (((quadrant + 1u) & 2u) != 0u) cs = -cs;  // quadrants 1, 2
    if ((quadrant & 2u) != 0u) sn = -sn;         // quadrants 2, 3
    return make_float2(cs, sn);
}

template <typename T> __device__ __forceinline__ uint4 narrow_chunk(const float *f);
template <> __device__ __forceinline__ uint4 narrow_chunk<float>(const float *f)
{
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <> __device__ __forceinline__ uint4 narrow_chunk<__nv_bfloat16>(const float *f)
{
    return make_uint4(pack_pair<__nv_bfloat16>(f[0], f[1]), pack_pair<__nv_bfloat16>(f[2], f[3]),
                      pack_pair<__nv_bfloat16>(f[4], f[5]), pack_pair<__nv_bfloat16>(f[6], f[7]));
}
template <> __device__ __forceinline__ uint4 narrow_chunk<__half>(const float *f)
{
    return make_uint4(pack_pair<__half>(f[0], f[1]), pack_pair<__half>(f[2], f[3]), pack_pair<__half>(f[4], f[5]),
                      pack_pair<__half>(f[6], f[7]));
}

// One unit of a token: where it is read and written, and its first frequency
// (-1: a plain copy of one chunk).  second: chunks to the pair's other chunk
// (0: one chunk only).
struct RopeUnit {
    const uint4 *src;
    uint4 *dst;  // null: nothing is written
    int freq, second;
};

// The token's rows in head 0 (chunk 0), and chunks between heads in the caches.
struct RopeToken {
    const uint4 *q, *k_new, *v_new;
    uint4 *q_out, *k_cache, *v_cache;  // (caches null: the page is not in the pool)
    long long cache_head;
};

template <typename T, bool kNeighbours>
__device__ __forceinline__ RopeUnit rope_unit(const RopeArgs &a, const RopeToken &tok, int u)
{
    constexpr int E = Elem<T>::kPerChunk;
    RopeUnit r;
    const int turned = (a.H_q + a.H_kv) * a.row_units;
    int row, c;
    if (u < turned) {
        row = quotient_of(u, a.inv_row_units);
        const int k = u - row * a.row_units;
        if (k < a.rot_units) {
            c = k;
            r.freq = k * (kNeighbours ? E / 2 : E);
            r.second = kNeighbours ? 0 : a.rot_units;
        } else {
            c = k + (kNeighbours ? 0 : a.rot_units);  // (halves: rot_units chunk pairs come first)
            r.freq = -1;
            r.second = 0;
        }
    } else {
        const int h = quotient_of(u - turned, a.inv_row_chunks);
        row = a.H_q + a.H_kv + h;
        c = u - turned - h * a.row_chunks;
        r.freq = -1;
        r.second = 0;
    }
    if (row < a.H_q) {
        r.src = tok.q + (row * a.sq[1] + c);
        r.dst = tok.q_out + ((long long)row * a.N * a.row_chunks + c);
    } else {
        const bool key = row < a.H_q + a.H_kv;
        const int h = row - a.H_q - (key ? 0 : a.H_kv);
        r.src = (key ? tok.k_new : tok.v_new) + (h * (key ? a.sk[1] : a.sv[1]) + c);
        uint4 *cache = key ? tok.k_cache : tok.v_cache;
        r.dst = cache == nullptr ? nullptr : cache + (h * tok.cache_head + c);
    }
    return r;
}

template <typename T, bool kNeighbours>
__device__ __forceinline__ void rope_store(const RopeUnit &r, const uint4 &x, const uint4 &y, const float2 *turn)
{
    constexpr int E = Elem<T>::kPerChunk;
    if (r.dst == nullptr) return;
    if (r.freq < 0) {
        stg128(r.dst, x);
        return;
    }
    if constexpr (kNeighbours) {
        float f[E];
        Elem<T>::widen(x, f);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 t = turn[r.freq + e / 2];
            const float p = f[e], q = f[e + 1];
            f[e] = fmaf(p, t.x, -(q * t.y));
            f[e + 1] = fmaf(p, t.y, q * t.x);
        }
        stg128(r.dst, narrow_chunk<T>(f));
    } else {
        float p[E], q[E];
        Elem<T>::widen(x, p);
        Elem<T>::widen(y, q);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 t = turn[r.freq + e];
            const float a = p[e], b = q[e];
            p[e] = fmaf(a, t.x, -(b * t.y));
            q[e] = fmaf(a, t.y, b * t.x);
        }
        stg128(r.dst, narrow_chunk<T>(p));
        stg128(r.dst + r.second, narrow_chunk<T>(q));
    }
}

// (q_out may be q itself: a unit is read before it is written, by one thread,
// and units do not overlap; so no load here is a read-only-cache load of q)
__device__ __forceinline__ uint4 ldg128(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

constexpr int kRopeThreads = 256;

template <typename T, bool kNeighbours>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs a)
{
    extern __shared__ float2 turn[];  // cos, sin of the token's n_freq angles
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = (int)(blockIdx.x / (unsigned)a.N), i = (int)(blockIdx.x % (unsigned)a.N);
    const int P = __ldg(a.past_len + b);
    const int capacity = a.block_table != nullptr ? a.max_pages << a.page_shift : a.T_max;
    if (!past_len_ok(P, a.N, capacity, a.max_past_len)) {  // (the whole block)
        if (threadIdx.x == 0 && i == 0 && blockIdx.y == 0) raise_error(a.err_word, KVD_DEVERR_PAST_LEN);
        return;
    }
    const int t = P + i;
    long long slot_row, head_rows;  // cache row of the token in head 0, and rows per head
    if (a.block_table != nullptr) {
        const int page = __ldg(a.block_table + (size_t)b * a.max_pages + (t >> a.page_shift));
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok && threadIdx.x == 0 && blockIdx.y == 0) raise_error(a.err_word, KVD_DEVERR_PAGE);
        head_rows = 1ll << a.page_shift;
        slot_row = ok ? (long long)page * a.H_kv * head_rows + (t & ((1 << a.page_shift) - 1)) : -1;
    } else {
        head_rows = a.T_max;
        slot_row = (long long)b * a.H_kv * head_rows + t;
    }

    RopeToken tok;
    tok.q = a.q + (b * a.sq[0] + i * a.sq[2]);
    tok.k_new = a.k_new + (b * a.sk[0] + i * a.sk[2]);
    tok.v_new = a.v_new + (b * a.sv[0] + i * a.sv[2]);
    tok.q_out = a.q_out + ((long long)b * a.H_q * a.N + i) * a.row_chunks;
    tok.k_cache = slot_row < 0 ? nullptr : a.k_cache + slot_row * a.row_chunks;
    tok.v_cache = slot_row < 0 ? nullptr : a.v_cache + slot_row * a.row_chunks;
    tok.cache_head = head_rows * a.row_chunks;

    const int u_end = min(a.units, (int)(blockIdx.y + 1) * a.split_units);
    int u = (int)blockIdx.y * a.split_units + (int)threadIdx.x;
    RopeUnit r[2];
    uint4 x[2], y[2];
    auto load = [&](int k, int uk) {
        r[k].dst = nullptr;
        if (uk >= u_end) return;
        r[k] = rope_unit<T, kNeighbours>(a, tok, uk);
        x[k] = ldg128(r[k].src);
        if (r[k].second) y[k] = ldg128(r[k].src + r[k].second);
    };
    load(0, u);
    load(1, u + (int)blockDim.x);

    const int64_t pos = (int64_t)a.pos_base + (a.positions != nullptr ? (int64_t)__ldg(a.positions + (size_t)b * a.N + i)
                                                                      : (int64_t)t);
    for (int f = threadIdx.x; f < a.n_freq; f += blockDim.x) turn[f] = rotation_of(turns_from_radians(__ldg(a.inv_freq + f)), pos);
    __syncthreads();

    for (;;) {
        rope_store<T, kNeighbours>(r[0], x[0], y[0], turn);
        rope_store<T, kNeighbours>(r[1], x[1], y[1], turn);
        u += 2 * (int)blockDim.x;
        if (u >= u_end) break;
        load(0, u);
        load(1, u + (int)blockDim.x);
    }
}

using RopeKernel = void (*)(const RopeArgs);

RopeKernel pick_rope_kernel(kvd_dtype dtype, bool neighbours)
{
    switch (dtype) {
    case KVD_F32: return neighbours ? rope_append_kernel<float, true> : rope_append_kernel<float, false>;
    case KVD_BF16: return neighbours ? rope_append_kernel<__nv_bfloat16, true> : rope_append_kernel<__nv_bfloat16, false>;
    case KVD_F16: return neighbours ? rope_append_kernel<__half, true> : rope_append_kernel<__half, false>;
    default: return nullptr;
    }
}

constexpr int kRopeMaxD = 4096;  // the angles of a row in 16 KB of shared memory

kvd_status rope_launch(const void *q, void *q_out, void *k_cache, void *v_cache, const void *k_new, const void *v_new,
                       const int64_t *strides, const PagedCache *paged, const int32_t *past_len,
                       const int32_t *positions, int pos_base, const double *inv_freq, int rot_dim, int interleaved,
                       int B, int H_q, int H_kv, int T_max, int D, int N, int max_past_len, kvd_dtype dtype,
                       uint32_t *err_word, void *stream)
{
    if (dtype != KVD_F32 && dtype != KVD_BF16 && dtype != KVD_F16) return KVD_ERR_UNSUPPORTED;
    const int es = elem_bytes(dtype), E = 16 / es;
    if (!q || !q_out || !k_cache || !v_cache || !k_new || !v_new || !past_len || !inv_freq) return KVD_ERR_INVALID_ARG;
    if (B < 0 || H_q < 1 || H_kv < 1 || D < 1 || N < 1 || max_past_len < 0) return KVD_ERR_INVALID_ARG;
    if (rot_dim < 2 || rot_dim > D || rot_dim % 2 != 0) return KVD_ERR_INVALID_ARG;
    int page_shift = 0;
    if (paged != nullptr) {
        const kvd_status st = check_paged(*paged, &T_max, &page_shift);
        if (st != KVD_OK) return st;
    }
    if (T_max < 1) return KVD_ERR_INVALID_ARG;
    if (D % E != 0 || D > kRopeMaxD || rot_dim % (interleaved ? E : 2 * E) != 0) return KVD_ERR_UNSUPPORTED;
    for (const void *p : {q, (const void *)q_out, (const void *)k_cache, (const void *)v_cache, k_new, v_new})
        if (!aligned16(p)) return KVD_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0) return KVD_ERR_INVALID_ARG;
    if (strides != nullptr)
        for (int k = 0; k < 9; ++k)
            if (strides[k] < 0 || strides[k] % E != 0) return KVD_ERR_INVALID_ARG;
    if ((long long)max_past_len + N > T_max) return KVD_ERR_CAPACITY;
    if (B == 0) return KVD_OK;
    const long long tokens = (long long)B * N;
    const int row_chunks = D / E;
    const int rot_units = rot_dim / E / (interleaved ? 1 : 2);
    const int row_units = rot_units + (D - rot_dim) / E;
    const long long units = ((long long)H_q + H_kv) * row_units + (long long)H_kv * row_chunks;
    if (tokens > 0x7fffffffLL || units >= kRopeMaxUnits) return KVD_ERR_UNSUPPORTED;

    int sms = 0;
    const kvd_status st = current_sm_count(&sms);
    if (st != KVD_OK) return st;

    RopeArgs a;
    a.q = static_cast<const uint4 *>(q);
    a.k_new = static_cast<const uint4 *>(k_new);
    a.v_new = static_cast<const uint4 *>(v_new);
    a.q_out = static_cast<uint4 *>(q_out);
    a.k_cache = static_cast<uint4 *>(k_cache);
    a.v_cache = static_cast<uint4 *>(v_cache);
    a.past_len = past_len;
    a.positions = positions;
    a.block_table = paged != nullptr ? paged->block_table : nullptr;
    a.inv_freq = inv_freq;
    a.err_word = err_word;
    const long long dq[3] = {(long long)H_q * N * row_chunks, (long long)N * row_chunks, row_chunks};
    const long long dk[3] = {(long long)H_kv * N * row_chunks, (long long)N * row_chunks, row_chunks};
    for (int k = 0; k < 3; ++k) {
        a.sq[k] = strides != nullptr ? strides[k] / E : dq[k];
        a.sk[k] = strides != nullptr ? strides[3 + k] / E : dk[k];
        a.sv[k] = strides != nullptr ? strides[6 + k] / E : dk[k];
    }
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.N = N;
    a.T_max = T_max;
    a.max_past_len = max_past_len;
    a.page_shift = page_shift;
    a.max_pages = paged != nullptr ? paged->max_pages : 0;
    a.num_pages = paged != nullptr ? paged->num_pages : 0;
    a.pos_base = pos_base;
    a.n_freq = rot_dim / 2;
    a.row_chunks = row_chunks;
    a.rot_units = rot_units;
    a.row_units = row_units;
    a.units = (int)units;
    a.inv_row_units = ((1ull << 36) + row_units - 1) / row_units;
    a.inv_row_chunks = ((1ull << 36) + row_chunks - 1) / row_chunks;

    // Fewer tokens than SMs: a token's units are shared out over several
    // blocks (at least 64 units each, so that the angles are not most of it).
    long long splits = 1;
    if (tokens < sms) {
        splits = (sms + tokens - 1) / tokens;
        const long long most = (units + 63) / 64;
        if (splits > most) splits = most;
    }
    a.split_units = (int)((units + splits - 1) / splits);
    // as many threads as make the passes over a block's units even
    const int passes = (a.split_units + kRopeThreads - 1) / kRopeThreads;
    const int threads = ((a.split_units + passes - 1) / passes + 31) / 32 * 32;

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tokens, (unsigned)splits);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)a.n_freq * sizeof(float2);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {&a};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(pick_rope_kernel(dtype, interleaved != 0)), args) ==
                   cudaSuccess
               ? KVD_OK
               : KVD_ERR_CUDA;
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" {

kvd_status kvd_rope_append(const void *q, void *q_out, void *k_cache, void *v_cache, const void *k_new,
                           const void *v_new, const int64_t *strides, const int32_t *past_len,
                           const int32_t *positions, int pos_base, const double *inv_freq, int rot_dim,
                           int interleaved, int B, int H_q, int H_kv, int T_max, int D, int N, int max_past_len,
                           kvd_dtype dtype, uint32_t *err_word, void *stream)
{
    return rope_launch(q, q_out, k_cache, v_cache, k_new, v_new, strides, nullptr, past_len, positions, pos_base,
                       inv_freq, rot_dim, interleaved, B, H_q, H_kv, T_max, D, N, max_past_len, dtype, err_word, stream);
}

kvd_status kvd_paged_rope_append(const void *q, void *q_out, void *k_pages, void *v_pages, const void *k_new,
                                 const void *v_new, const int64_t *strides, const int32_t *block_table,
                                 const int32_t *past_len, const int32_t *positions, int pos_base,
                                 const double *inv_freq, int rot_dim, int interleaved, int B, int H_q, int H_kv, int D,
                                 int N, int page_size, int max_pages, int num_pages, int max_past_len, kvd_dtype dtype,
                                 uint32_t *err_word, void *stream)
{
    const PagedCache pc{block_table, page_size, max_pages, num_pages};
    return rope_launch(q, q_out, k_pages, v_pages, k_new, v_new, strides, &pc, past_len, positions, pos_base, inv_freq,
                       rot_dim, interleaved, B, H_q, H_kv, 0, D, N, max_past_len, dtype, err_word, stream);
}

}  // extern "C"
