// cache.hip -- keys and values into 4-bit pages and back on gfx950.
//
// A group of 32 channels x becomes s = up5(max |x| / 7), c = rne(x / s): up5 rounds up to 5
// significant bits, so |x / s| <= 7, and c s (3 bits times 5) is exact in bf16.  The codes are those
// of the exact quotient: the kernel takes rint(x * (1 / s)) and moves it by one where the remainder
// x - c s, which is exact in f32, passes s / 2 (or equals it and c is odd).
//
// One workgroup per row of the call (its place is looked up once).  Keys: a lane holds 8
// neighbouring channels, which are one word of the key row, four lanes a group.  Values: a lane
// holds channel m of every 16, so that its nibbles are the bytes it stores.
#include "cache.hpp"

namespace gptq {

constexpr int kCacheThreads = 256;

struct CacheArgs {
    CacheView c;
    Batch q;
    const void* K;
    const void* V;
    int64_t ld, ldh;
};
struct CacheOut {
    CacheView c;
    Batch q;
    void* K;
    void* V;
    int64_t ld, ldh;
};

// s of a group from its largest magnitude (the bits of |x| compare as unsigned, NaN above all).
__device__ __forceinline__ float group_scale(uint32_t top) {
    if (top == 0u) return 0.0f;
    if (top >= 0x7f000000u) return __uint_as_float(0x7fc00000u);  // 2^127 and above, inf, NaN
    const double a = (double)__uint_as_float(top) / 7.0;
    uint64_t b = (uint64_t)__double_as_longlong(a);
    b = (b + ((1ull << 48) - 1)) & ~((1ull << 48) - 1);
    return (float)fmax(__longlong_as_double((long long)b), 0x1p-126);
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The code + 8 of one value; inv = 1 / s, or 0 where s is 0 or NaN.
__device__ __forceinline__ uint32_t code_of(float x, float s, float inv) {
    float c = rintf(x * inv);
    const float r = fmaf(-c, s, x), half = 0.5f * s;
    const bool odd = ((int)c & 1) != 0;
    if (r > half || (r == half && odd)) c += 1.0f;
    if (r < -half || (r == -half && odd)) c -= 1.0f;
    return inv == 0.0f ? 8u : (uint32_t)((int)c + 8);
}
__device__ __forceinline__ float inverse(float s) { return s > 0.0f ? 1.0f / s : 0.0f; }

template <int DT, int G>
__global__ __launch_bounds__(kCacheThreads) void cache_write_kernel(CacheArgs a) {
    const int row = blockIdx.x, tid = threadIdx.x;
    const int b = seq_of_row(a.q, row);
    if (b < 0) return;
    int r0, r1;
    seq_rows(a.q, b, r0, r1);
    const int64_t pos = (int64_t)a.q.len[b] - (r1 - r0) + (row - r0);
    const int64_t place = cache_row(a.c, a.q, b, pos, 0);
    if (place < 0) return;
    // Keys: lane (head, i, h) takes channels 32 i + 8 h .. + 7.
    for (int u = tid; u < a.c.heads * G * 4; u += kCacheThreads) {
        const int head = u / (4 * G), i = (u >> 2) % G, h = u & 3;
        float x[8];
        load_eight<DT>(a.K, (int64_t)row * a.ld + head * a.ldh + 32 * i + 8 * h, x);
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, magnitude(x[k]));
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const float s = group_scale(top), inv = inverse(s);
        uint32_t w = 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w |= code_of(x[2 * k], s, inv) << (4 * k) | code_of(x[2 * k + 1], s, inv) << (4 * k + 16);
        const int64_t at = place + (int64_t)head * a.c.page;
        *(uint32_t*)(a.c.k + at * (16 * G) + 4 * (h * G + i)) = w;
        if (h == 0) a.c.ks[at * G + i] = (uint16_t)(__float_as_uint(s) >> 16);
    }
    // Values: lane (head, m) takes channels m + 16 j.
    for (int u = tid; u < a.c.heads * 16; u += kCacheThreads) {
        const int head = u >> 4, m = u & 15;
        const int64_t at = place + (int64_t)head * a.c.page;
        uint32_t w[(G + 3) / 4] = {};
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int64_t e = (int64_t)row * a.ld + head * a.ldh + 32 * i + m;
            const float x0 = load_one<DT>(a.V, e), x1 = load_one<DT>(a.V, e + 16);
            uint32_t top = max(magnitude(x0), magnitude(x1));
#pragma unroll
            for (int k = 1; k < 16; k *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, k));
            const float s = group_scale(top), inv = inverse(s);
            w[i >> 2] |= (code_of(x0, s, inv) | code_of(x1, s, inv) << 4) << (8 * (i & 3));
            if (m == 0) a.c.vs[at * G + i] = (uint16_t)(__float_as_uint(s) >> 16);
        }
        uint8_t* p = a.c.v + at * (16 * G) + m * G;
        if constexpr (G == 2) *(uint16_t*)p = (uint16_t)w[0];
        if constexpr (G == 4) *(uint32_t*)p = w[0];
        if constexpr (G == 8) *(u32v2*)p = u32v2{w[0], w[1]};
    }
}

__device__ __forceinline__ float code_value(uint32_t nibble, float s) { return (float)((int)nibble - 8) * s; }
template <int DT>
__device__ __forceinline__ float saturate(float v) {
    if constexpr (DT == GPTQ_F16) {
        if (v > 65504.0f) v = 65504.0f;  // NaN stays
        if (v < -65504.0f) v = -65504.0f;
    }
    return v;
}

template <int DT, int G>
__global__ __launch_bounds__(kCacheThreads) void cache_read_kernel(CacheOut a) {
    const int row = blockIdx.x, tid = threadIdx.x;
    const int b = seq_of_row(a.q, row);
    if (b < 0) return;
    int r0, r1;
    seq_rows(a.q, b, r0, r1);
    const int64_t pos = (int64_t)a.q.len[b] - (r1 - r0) + (row - r0);
    const int64_t place = cache_row(a.c, a.q, b, pos, 0);
    // Lane (head, i, h) writes channels 32 i + 8 h .. + 7 of keys and values.
    for (int u = tid; u < a.c.heads * G * 4; u += kCacheThreads) {
        const int head = u / (4 * G), i = (u >> 2) % G, h = u & 3;
        const int64_t at = place + (int64_t)head * a.c.page, e = (int64_t)row * a.ld + head * a.ldh + 32 * i + 8 * h;
        if (a.K) {
            const uint32_t w = place < 0 ? 0u : *(const uint32_t*)(a.c.k + at * (16 * G) + 4 * (h * G + i));
            const float s = place < 0 ? 0.0f : __uint_as_float((uint32_t)a.c.ks[at * G + i] << 16);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = saturate<DT>(code_value((w >> (4 * (2 * k + (j >> 1)) + 16 * (j & 1))) & 15u, s));
                store_four<DT>(a.K, e + 4 * k, v);
            }
        }
        if (a.V) {
            const float s = place < 0 ? 0.0f : __uint_as_float((uint32_t)a.c.vs[at * G + i] << 16);
            const uint8_t* p = a.c.v + at * (16 * G) + (8 * (h & 1)) * G + i;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t byte = place < 0 ? 0u : p[(4 * k + j) * G];
                    v[j] = saturate<DT>(code_value((byte >> (4 * (h >> 1))) & 15u, s));
                }
                store_four<DT>(a.V, e + 4 * k, v);
            }
        }
    }
}

template <template <int, int> class F, class Fn>
struct Pick {
    static Fn get(int dt, int dim) {
        switch (dt) {
            case GPTQ_F32: return dim == 64 ? F<GPTQ_F32, 2>::fn : dim == 128 ? F<GPTQ_F32, 4>::fn : F<GPTQ_F32, 8>::fn;
            case GPTQ_BF16: return dim == 64 ? F<GPTQ_BF16, 2>::fn : dim == 128 ? F<GPTQ_BF16, 4>::fn : F<GPTQ_BF16, 8>::fn;
            default: return dim == 64 ? F<GPTQ_F16, 2>::fn : dim == 128 ? F<GPTQ_F16, 4>::fn : F<GPTQ_F16, 8>::fn;
        }
    }
};
typedef void (*WriteKernel)(CacheArgs);
typedef void (*ReadKernel)(CacheOut);
template <int DT, int G>
struct WriteFn {
    static constexpr WriteKernel fn = cache_write_kernel<DT, G>;
};
template <int DT, int G>
struct ReadFn {
    static constexpr ReadKernel fn = cache_read_kernel<DT, G>;
};

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_cache_write(const gptq_cache* cache, const gptq_batch* batch, const void* K, const void* V,
                                int64_t ld, int64_t ldh, int dtype, void* stream) {
    const int es = dtype_size(dtype);
    if (!es || !cache_ok(cache) || !batch_ok(batch)) return GPTQ_EINVAL;
    if (batch->rows == 0) return GPTQ_OK;
    if (!K || !V || !heads_ok(K, batch->rows, ld, ldh, cache->heads, cache->dim, es) ||
        !heads_ok(V, batch->rows, ld, ldh, cache->heads, cache->dim, es))
        return GPTQ_EINVAL;
    CheckScope check;
    check_cache(cache, batch);
    const size_t bytes = heads_bytes(batch->rows, ld, ldh, cache->heads, cache->dim, es);
    check_buffer(K, bytes, "K");
    check_buffer(V, bytes, "V");
    hipStream_t st = (hipStream_t)stream;
    const CacheArgs a{cache_view(cache), batch_view(batch), K, V, ld, ldh};
    const WriteKernel k = Pick<WriteFn, WriteKernel>::get(dtype, cache->dim);
    const int64_t dense = (int64_t)cache->heads * cache->dim, wide = (cache->heads - 1) * ldh + cache->dim;
    {
        ProfScope ps(FAM_CACHE, st, 0.0, (double)batch->rows * dense * (2.0 * es + 1.125));
        GPTQ_LAUNCH(st, "cache_write", (k<<<(unsigned)batch->rows, kCacheThreads, 0, st>>>(a)),
                    rd(K, ld, batch->rows, wide, es), rd(V, ld, batch->rows, wide, es), batch_span(batch, 0),
                    batch_span(batch, 1), batch_span(batch, 2), plane(cache->k, cache, cache->dim / 2, true),
                    plane(cache->v, cache, cache->dim / 2, true), plane(cache->k_scale, cache, cache->dim / 16, true),
                    plane(cache->v_scale, cache, cache->dim / 16, true));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}

extern "C" int gptq_cache_read(const gptq_cache* cache, const gptq_batch* batch, void* K, void* V, int64_t ld,
                               int64_t ldh, int dtype, void* stream) {
    const int es = dtype_size(dtype);
    if (!es || !cache_ok(cache) || !batch_ok(batch)) return GPTQ_EINVAL;
    if (batch->rows == 0) return GPTQ_OK;
    if ((!K && !V) || !heads_ok(K, batch->rows, ld, ldh, cache->heads, cache->dim, es) ||
        !heads_ok(V, batch->rows, ld, ldh, cache->heads, cache->dim, es))
        return GPTQ_EINVAL;
    CheckScope check;
    check_cache(cache, batch);
    const size_t bytes = heads_bytes(batch->rows, ld, ldh, cache->heads, cache->dim, es);
    if (K) check_buffer(K, bytes, "K");
    if (V) check_buffer(V, bytes, "V");
    hipStream_t st = (hipStream_t)stream;
    const CacheOut a{cache_view(cache), batch_view(batch), K, V, ld, ldh};
    const ReadKernel k = Pick<ReadFn, ReadKernel>::get(dtype, cache->dim);
    const int64_t dense = (int64_t)cache->heads * cache->dim, wide = (cache->heads - 1) * ldh + cache->dim;
    {
        ProfScope ps(FAM_CACHE, st, 0.0, (double)batch->rows * dense * (2.0 * es + 1.125));
        GPTQ_LAUNCH(st, "cache_read", (k<<<(unsigned)batch->rows, kCacheThreads, 0, st>>>(a)),
                    batch_span(batch, 0), batch_span(batch, 1), batch_span(batch, 2),
                    plane(cache->k, cache, cache->dim / 2, false), plane(cache->v, cache, cache->dim / 2, false),
                    plane(cache->k_scale, cache, cache->dim / 16, false),
                    plane(cache->v_scale, cache, cache->dim / 16, false),
                    wr(K ? K : V, ld, K ? batch->rows : 0, wide, es), wr(V ? V : K, ld, V ? batch->rows : 0, wide, es));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}
