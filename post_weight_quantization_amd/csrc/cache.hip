// cache.hip -- keys and values into 4-bit pages and back on gfx950.
//
// A group of 32 channels x becomes s = up5(max |x| / 7), c = rne(x / s): up5 rounds up to 5
// significant bits, so |x / s| <= 7, and c s (3 bits times 5) is exact in bf16.  Both are exact: s is
// the smallest such number with 7 s >= max |x| (8 bits, exact in f32), looked for from an estimate;
// c is the correctly rounded quotient's (see encode).
//
// A workgroup takes up to 8 rows of the call.  Their places are looked up first, side by side, and kept in
// LDS; then a lane holds 8 neighbouring channels of a row and head, four lanes a group, and reads and
// writes 16 bytes of the dense side.  Those channels are one word of a key's row; of a value's row they are
// nibbles of 8 bytes G apart, which go by way of LDS when written and are picked from 8 G loaded bytes
// when read.
//
// Both are bound by memory: 6 x up to 4096 rows (10 heads of 64, f16) are written in 15 us, 4.0 TB/s of 16-bit
// rows and codes, and read back in 15; 8 x up to 8192 rows (8 heads of 128, bf16) are read in 66 us, 4.3 TB/s.
// 48 single rows take 3.4 and 3.1 us, a launch.  One row a workgroup wrote those prompts in 45 us, most of
// it in the search for its place; codes by the remainder of a rounded product, not of the quotient,
// in 24, most of it vector instructions.
#include "cache.hpp"

namespace gptq {

constexpr int kCacheThreads = 256, kCacheRows = 8;

struct CacheArgs {
    CacheView c;
    Batch q;
    const void* K;
    const void* V;
    int64_t ld, ldh;
    int rows;  // of a workgroup, up to kCacheRows
};
struct CacheOut {
    CacheView c;
    Batch q;
    void* K;
    void* V;
    int64_t ld, ldh;
    int rows;
};

// Places (cache rows of head 0) of the workgroup's n rows from row0 on: -1 where there is none, -2 for a row
// of no sequence.  Lane i of the first wave finds row i's.
__device__ __forceinline__ void find_places(const CacheView& c, const Batch& q, int row0, int n, int64_t* place) {
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x, row = row0 + lane;
        int b = row;
        if (q.start) {
            // Sequences that end at or before the row.
            if (q.seqs <= 64) {
                const int end = lane < q.seqs ? q.start[lane + 1] : 0x7fffffff;
                b = 0;
                for (int i = 0; i < n; ++i) {
                    const int before = __popcll(__ballot(end <= row0 + i));
                    if (lane == i) b = before;
                }
                if (row < q.start[0]) b = -1;
            } else {
                int lo = 0, hi = q.seqs;  // the first sequence of those that end behind the row
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (q.start[mid + 1] > row)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                b = row < q.start[0] ? -1 : lo;
            }
        }
        if (lane < n) {
            int64_t at = -2;
            if (b >= 0 && b < q.seqs) {
                int r0, r1;
                seq_rows(q, b, r0, r1);
                at = cache_row(c, q, b, (int64_t)q.len[b] - (r1 - r0) + (row - r0), 0);
            }
            place[lane] = at;
        }
    }
    __syncthreads();
}

// s of a group from its largest magnitude (the bits of |x| compare as unsigned, NaN above all).
__device__ __forceinline__ float group_scale(uint32_t top) {
    const float a = __uint_as_float(top);
    // A little below a / 7, cut to 5 bits: the answer is this or one of the next two.
    uint32_t b = __float_as_uint(a * 0x1.249248p-3f) & 0xfff80000u;
#pragma unroll
    for (int k = 0; k < 2; ++k) b += 7.0f * __uint_as_float(b) < a ? 0x00080000u : 0u;
    float s = fmaxf(__uint_as_float(b), 0x1p-126f);
    if (top == 0u) s = 0.0f;
    if (top >= 0x7f000000u) s = __uint_as_float(0x7fc00000u);  // 2^127 and above, inf, NaN
    return s;
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Codes of the 8 values a lane holds, as whole floats, and their group's scale (its other values are in the
// next three lanes).  The quotient x / s is the correctly rounded one: from a correctly rounded 1 / s (a
// Newton step on the reciprocal, whose error of one unit it needs; s is not all ones) the product q and one
// step by its remainder, which is exact, round as the quotient does.  That cannot land on a half that
// x / s is not: halves times s have 9 bits, so the next x is a whole unit away.  A group with a tiny scale
// is lifted by 2^64 first, so that remainders stay normal.
__device__ __forceinline__ float encode(const float (&x)[8], float (&code)[8]) {
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, magnitude(x[k]));
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const float scale = group_scale(top);
    float s = scale, z[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = x[k];
    const bool tiny = s < 0x1p-60f;
    if (__ballot(tiny)) {
        const float lift = tiny ? 0x1p64f : 1.0f;
        s *= lift;
#pragma unroll
        for (int k = 0; k < 8; ++k) z[k] *= lift;
    }
    float inv = __builtin_amdgcn_rcpf(s);
    inv = fmaf(fmaf(-s, inv, 1.0f), inv, inv);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float q = z[k] * inv;
        code[k] = rintf(fmaf(fmaf(-q, s, z[k]), inv, q));
    }
    return scale;
}
// Four codes' nibbles (+ 8), the first lowest, exact in f32.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    return (uint32_t)fmaf(d, 4096.0f, fmaf(c, 256.0f, fmaf(b, 16.0f, a + 34952.0f)));
}
// Eight nibbles, all 8 (code 0) where the scale is 0 or NaN.
__device__ __forceinline__ uint32_t pack8(uint32_t low, uint32_t high, float s) {
    return s > 0.0f ? low | high << 16 : 0x88888888u;
}

template <int DT, int G>
__global__ __launch_bounds__(kCacheThreads) void cache_write_kernel(CacheArgs a) {
    __shared__ int64_t place[kCacheRows];
    __shared__ __attribute__((aligned(16))) uint8_t stage[kCacheThreads / (4 * G)][16 * G];
    const int row0 = blockIdx.x * a.rows, n = min(a.rows, (int)a.q.rows - row0);
    find_places(a.c, a.q, row0, n, place);
    const int i = (threadIdx.x >> 2) % G, h = threadIdx.x & 3, slot = threadIdx.x / (4 * G);
    // All of a slot's lanes are in one wave and walk together: what they leave in LDS is theirs.
    for (int u = slot; u < n * a.c.heads; u += kCacheThreads / (4 * G)) {
        const int r = u / a.c.heads, head = u - r * a.c.heads;
        const int64_t at0 = place[r];
        if (at0 < 0) continue;
        const int64_t at = at0 + (int64_t)head * a.c.page;
        const int64_t e = (int64_t)(row0 + r) * a.ld + head * a.ldh + 32 * i + 8 * h;
        float x[8], y[8];
        load_eight<DT>(a.K, e, x);
        load_eight<DT>(a.V, e, y);
        float code[8];
        const float ks = encode(x, code);
        *(uint32_t*)(a.c.k + at * (16 * G) + 4 * (h * G + i)) =
            pack8(pack4(code[0], code[2], code[4], code[6]), pack4(code[1], code[3], code[5], code[7]), ks);
        const float vs = encode(y, code);
        if (h == 0) {
            a.c.ks[at * G + i] = (uint16_t)(__float_as_uint(ks) >> 16);
            a.c.vs[at * G + i] = (uint16_t)(__float_as_uint(vs) >> 16);
        }
        // Channel 32 i + m shares a byte with 32 i + 16 + m, two lanes on.
        const uint32_t w = pack8(pack4(code[0], code[1], code[2], code[3]), pack4(code[4], code[5], code[6], code[7]), vs);
        const uint32_t other = (uint32_t)__shfl_xor((int)w, 2);
        const uint32_t lo = h < 2 ? w : other, hi = h < 2 ? other : w;
        // The lower of the two lanes makes the even bytes, the upper one the odd.
        const uint32_t bytes = h < 2 ? (lo & 0x0f0f0f0fu) | (hi & 0x0f0f0f0fu) << 4 : (lo >> 4 & 0x0f0f0f0fu) | (hi & 0xf0f0f0f0u);
#pragma unroll
        for (int k = 0; k < 4; ++k) stage[slot][(8 * (h & 1) + 2 * k + (h >> 1)) * G + i] = (uint8_t)(bytes >> (8 * k));
        __builtin_amdgcn_wave_barrier();
        const int l = threadIdx.x % (4 * G);  // 4 bytes a lane
        *(uint32_t*)(a.c.v + at * (16 * G) + 4 * l) = *(const uint32_t*)&stage[slot][4 * l];
        __builtin_amdgcn_wave_barrier();
    }
}

template <int DT>
__device__ __forceinline__ float saturate(float v) {
    if constexpr (DT == GPTQ_F16) {
        if (v > 65504.0f) v = 65504.0f;  // NaN stays
        if (v < -65504.0f) v = -65504.0f;
    }
    return v;
}
template <int DT>
__device__ __forceinline__ void store_values(void* p, int64_t e, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = saturate<DT>(v[k]);
    if constexpr (DT == GPTQ_F32) {
        *(f32v4*)((float*)p + e) = f32v4{v[0], v[1], v[2], v[3]};
        *(f32v4*)((float*)p + e + 4) = f32v4{v[4], v[5], v[6], v[7]};
    } else {
        store_eight<DT>(p, e, v);
    }
}

template <int DT, int G>
__global__ __launch_bounds__(kCacheThreads) void cache_read_kernel(CacheOut a) {
    __shared__ int64_t place[kCacheRows];
    const int row0 = blockIdx.x * a.rows, n = min(a.rows, (int)a.q.rows - row0);
    find_places(a.c, a.q, row0, n, place);
    const int i = (threadIdx.x >> 2) % G, h = threadIdx.x & 3;
    for (int u = threadIdx.x / (4 * G); u < n * a.c.heads; u += kCacheThreads / (4 * G)) {
        const int r = u / a.c.heads, head = u - r * a.c.heads;
        const int64_t at0 = place[r];
        if (at0 == -2) continue;
        const int64_t at = (at0 < 0 ? 0 : at0) + (int64_t)head * a.c.page;  // a place that does not exist reads as 0
        const int64_t e = (int64_t)(row0 + r) * a.ld + head * a.ldh + 32 * i + 8 * h;
        uint32_t kw = 0u, w[2 * G] = {};
        float ks = 0.0f, vs = 0.0f;
        if (at0 >= 0) {
            kw = *(const uint32_t*)(a.c.k + at * (16 * G) + 4 * (h * G + i));
            ks = __uint_as_float((uint32_t)a.c.ks[at * G + i] << 16);
            vs = __uint_as_float((uint32_t)a.c.vs[at * G + i] << 16);
#pragma unroll
            for (int k = 0; k < G / 2; ++k) {
                const u32v4 x = ((const u32v4*)(a.c.v + at * (16 * G) + 8 * G * (h & 1)))[k];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * k + j] = x[j];
            }
        }
        float v[8];
        if (a.K) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = (float)((int)(kw >> (4 * (k >> 1) + 16 * (k & 1)) & 15u) - 8) * ks;
            store_values<DT>(a.K, e, v);
        }
        if (a.V) {
            // Byte i of each G, of channel m = 8 (h % 2) + k; its nibble h / 2.
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t x = 0u;
                if constexpr (G == 2) x = w[k >> 1] >> (8 * i + 16 * (k & 1));
                if constexpr (G == 4) x = w[k] >> (8 * i);
                if constexpr (G == 8) {
                    const uint32_t w0 = w[2 * k], w1 = w[2 * k + 1];
                    x = (i & 4 ? w1 : w0) >> (8 * (i & 3));
                }
                v[k] = (float)((int)(x >> (4 * (h >> 1)) & 15u) - 8) * vs;
            }
            store_values<DT>(a.V, e, v);
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

// Rows of a workgroup: one while there are fewer than four workgroups a CU, then up to kCacheRows (prompts
// written and read 34.2 us with 8, 34.6 with 16, 37.3 with 32; 8 x up to 8192 tokens read 71.5, 74.0, 74.4).
static int cache_rows(int64_t rows) {
    const int64_t r = rows / 1024;
    return (int)(r < 1 ? 1 : r > kCacheRows ? kCacheRows : r);
}

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_cache_write(const gptq_cache* cache, const gptq_batch* batch, const void* K, const void* V,
                                int64_t ld, int64_t ldh, int dtype, void* stream) {
    const int es = dtype_size(dtype);
    if (!es || !cache_ok(cache) || !batch_ok(batch) || !table_ok(cache, batch)) return GPTQ_EINVAL;
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
    const CacheArgs a{cache_view(cache), batch_view(batch), K, V, ld, ldh, cache_rows(batch->rows)};
    const WriteKernel k = Pick<WriteFn, WriteKernel>::get(dtype, cache->dim);
    const int64_t dense = (int64_t)cache->heads * cache->dim, wide = (cache->heads - 1) * ldh + cache->dim;
    {
        ProfScope ps(FAM_CACHE, st, 0.0, (double)batch->rows * dense * (2.0 * es + 1.125));
        GPTQ_LAUNCH(st, "cache_write", (k<<<(unsigned)((batch->rows + a.rows - 1) / a.rows), kCacheThreads, 0, st>>>(a)),
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
    if (!es || !cache_ok(cache) || !batch_ok(batch) || !table_ok(cache, batch)) return GPTQ_EINVAL;
    if (batch->rows == 0) return GPTQ_OK;
    if (K == V || !heads_ok(K, batch->rows, ld, ldh, cache->heads, cache->dim, es) ||
        !heads_ok(V, batch->rows, ld, ldh, cache->heads, cache->dim, es))
        return GPTQ_EINVAL;
    const RowSet k_rows = heads_rows(K, batch->rows, ld, ldh, cache->heads, cache->dim, es),
                 v_rows = heads_rows(V, batch->rows, ld, ldh, cache->heads, cache->dim, es);
    if (rows_meet(k_rows, v_rows) || meets_cache(k_rows, cache) || meets_cache(v_rows, cache)) return GPTQ_EINVAL;
    CheckScope check;
    check_cache(cache, batch);
    const size_t bytes = heads_bytes(batch->rows, ld, ldh, cache->heads, cache->dim, es);
    if (K) check_buffer(K, bytes, "K");
    if (V) check_buffer(V, bytes, "V");
    hipStream_t st = (hipStream_t)stream;
    const CacheOut a{cache_view(cache), batch_view(batch), K, V, ld, ldh, cache_rows(batch->rows)};
    const ReadKernel k = Pick<ReadFn, ReadKernel>::get(dtype, cache->dim);
    const int64_t dense = (int64_t)cache->heads * cache->dim, wide = (cache->heads - 1) * ldh + cache->dim;
    {
        ProfScope ps(FAM_CACHE, st, 0.0, (double)batch->rows * dense * (2.0 * es + 1.125));
        GPTQ_LAUNCH(st, "cache_read", (k<<<(unsigned)((batch->rows + a.rows - 1) / a.rows), kCacheThreads, 0, st>>>(a)),
                    batch_span(batch, 0), batch_span(batch, 1), batch_span(batch, 2),
                    plane(cache->k, cache, cache->dim / 2, false), plane(cache->v, cache, cache->dim / 2, false),
                    plane(cache->k_scale, cache, cache->dim / 16, false),
                    plane(cache->v_scale, cache, cache->dim / 16, false),
                    wr(K ? K : V, ld, K ? batch->rows : 0, wide, es), wr(V ? V : K, ld, V ? batch->rows : 0, wide, es));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}
