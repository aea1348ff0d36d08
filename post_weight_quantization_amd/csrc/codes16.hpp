// codes16.hpp -- device helpers of the operators that multiply 4- and 2-bit codes on bf16 matrix
// units (linear.hip, cache.hip, attention.hip): element types, exact splits, code unpacking.
//
// A code is fed to v_mfma_f32_16x16x32_bf16 as the whole number it is: with the exponent of 16,
// 16 + q has q in bits 3..6 of bf16's mantissa, so a nibble becomes an operand by one shift and one
// and-or for two codes, exactly.  What 16 adds is taken out by the accumulator's start value: the
// same activations times a constant operand, one MFMA for all code tiles that share them.
//
// Lane layout of the 16x16x32 MFMA: A holds row lane % 16, B column lane % 16, both k = 8 (lane / 16)
// .. + 7 in four registers (two k each); D holds column lane % 16, rows 4 (lane / 16) .. + 3.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace gptq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32v4 __attribute__((ext_vector_type(4)));
typedef float f32v2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32v2 __attribute__((ext_vector_type(2)));

constexpr int kCUs = 256;

// Bytes of an element of a GPTQ_F32 / BF16 / F16 tensor; 0 for another value.
inline int dtype_size(int dt) { return dt == GPTQ_F32 ? 4 : (dt == GPTQ_BF16 || dt == GPTQ_F16) ? 2 : 0; }

// Rows of `bytes` bytes, `step` >= bytes apart.
struct RowSet {
    const void* p;
    int64_t step, rows, bytes;
};
inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }  // b > 0
// Do two sets share a byte?  Rows i of a and j of b meet where d - a.bytes < i a.step - j b.step < d + b.bytes.  With
// one step the least i - j above the first bound decides (slices of one buffer, whose ranges always
// meet); with two, rows of the shorter set are looked up in the other one by one, once their ranges meet.
inline bool rows_meet(RowSet a, RowSet b) {
    if (a.rows < 1 || b.rows < 1) return false;
    if (a.rows > b.rows) {
        const RowSet t = a;
        a = b;
        b = t;
    }
    const int64_t d = (int64_t)((intptr_t)b.p - (intptr_t)a.p);  // of b's first byte from a's
    if (a.rows == 1) a.step = b.step;
    const int64_t alen = (a.rows - 1) * a.step + a.bytes, blen = (b.rows - 1) * b.step + b.bytes;
    if (d >= alen || d + blen <= 0) return false;
    if (a.step == b.step) {
        int64_t k = floor_div(d - a.bytes, a.step) + 1;
        if (k < 1 - b.rows) k = 1 - b.rows;
        return k < a.rows && k * a.step < d + b.bytes;
    }
    for (int64_t i = 0; i < a.rows; ++i) {
        const int64_t at = i * a.step - d;  // of a's row i from b's first byte
        int64_t j = floor_div(at - b.bytes, b.step) + 1;
        if (j < 0) j = 0;
        if (j < b.rows && j * b.step < at + a.bytes) return true;
    }
    return false;
}

// Terms of bf16 (8 significant bits each) that hold a value of the type exactly.
template <int DT>
constexpr int kTerms = DT == GPTQ_BF16 ? 1 : DT == GPTQ_F16 ? 2 : 3;

__device__ __forceinline__ f32v4 mfma16(u32v4 a, u32v4 b, f32v4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Upper halves of two registers: (low half <- a, high half <- b).
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
__device__ __forceinline__ uint32_t pack_lo(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
// Two floats rounded to bf16, to nearest even (low half <- a).
__device__ __forceinline__ uint32_t round_bf16x2(float a, float b) {
    bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

template <int DT>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
    if constexpr (DT == GPTQ_F32) return ((const float*)p)[i];
    if constexpr (DT == GPTQ_BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
    if constexpr (DT == GPTQ_F16) return (float)((const _Float16*)p)[i];
}
template <int DT>
__device__ __forceinline__ void store_one(void* p, int64_t i, float v) {
    if constexpr (DT == GPTQ_F32) ((float*)p)[i] = v;
    if constexpr (DT == GPTQ_BF16) ((__bf16*)p)[i] = (__bf16)v;
    if constexpr (DT == GPTQ_F16) ((_Float16*)p)[i] = (_Float16)v;
}
// Eight elements as they lie in memory (16-byte aligned): four registers, eight in f32.
template <int DT>
struct Raw {
    u32v4 a[DT == GPTQ_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const char* q = (const char*)p + i * (DT == GPTQ_F32 ? 4 : 2);
        a[0] = *(const u32v4*)q;
        if constexpr (DT == GPTQ_F32) a[1] = *(const u32v4*)(q + 16);
    }
    __device__ __forceinline__ void floats(float (&v)[8]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t w = a[0][k];  // by value: a bit cast of a vector's element takes element 0
            if constexpr (DT == GPTQ_F32) {
                const uint32_t z = a[DT == GPTQ_F32][k];
                v[k] = __uint_as_float(w);
                v[k + 4] = __uint_as_float(z);
            } else if constexpr (DT == GPTQ_BF16) {
                v[2 * k] = __uint_as_float(w << 16);
                v[2 * k + 1] = __uint_as_float(w & 0xffff0000u);
            } else {
                typedef _Float16 h2 __attribute__((ext_vector_type(2)));
                const h2 x = __builtin_bit_cast(h2, w);
                v[2 * k] = (float)x[0];
                v[2 * k + 1] = (float)x[1];
            }
        }
    }
};
// Eight elements from element offset i as floats.
template <int DT>
__device__ __forceinline__ void load_eight(const void* p, int64_t i, float (&v)[8]) {
    Raw<DT> r;
    r.load(p, i);
    r.floats(v);
}
// Four elements stored as one vector (8- or 16-byte aligned address).
template <int DT>
__device__ __forceinline__ void store_four(void* p, int64_t i, const float (&v)[4]) {
    if constexpr (DT == GPTQ_F32) {
        *(f32v4*)((float*)p + i) = f32v4{v[0], v[1], v[2], v[3]};
    } else if constexpr (DT == GPTQ_BF16) {
        *(u32v2*)((uint16_t*)p + i) = u32v2{round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3])};
    } else {
        typedef _Float16 h4 __attribute__((ext_vector_type(4)));
        *(h4*)((uint16_t*)p + i) = h4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
    }
}

// Eight elements of a 16-bit type stored as one vector (16-byte aligned address).
template <int DT>
__device__ __forceinline__ void store_eight(void* p, int64_t i, const float* v) {
    u32v4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == GPTQ_BF16) {
            w[k] = round_bf16x2(v[2 * k], v[2 * k + 1]);
        } else {
            typedef _Float16 h2 __attribute__((ext_vector_type(2)));
            const h2 x = {(_Float16)v[2 * k], (_Float16)v[2 * k + 1]};
            w[k] = __builtin_bit_cast(uint32_t, x);
        }
    }
    *(u32v4*)((uint16_t*)p + i) = w;
}

// Eight elements as kTerms<DT> operands whose sum is the value exactly: each term takes the
// next 8 significant bits by truncation, and the differences are exact.  Register k holds
// elements (k, k + 4) with PAIR4, else (2 k, 2 k + 1).  raw: the elements as they lie in memory.
template <int DT, bool PAIR4 = true>
__device__ __forceinline__ void raw_terms(const u32v4* raw, u32v4 (&t)[kTerms<DT>]) {
    const u32v4 a = raw[0];
    if constexpr (DT == GPTQ_BF16) {
        if constexpr (PAIR4)
            t[0] = u32v4{pack_lo(a[0], a[2]), pack_hi(a[0], a[2]), pack_lo(a[1], a[3]), pack_hi(a[1], a[3])};
        else
            t[0] = a;
    } else {
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (DT == GPTQ_F32) {
                const u32v4 b = raw[1];
                v[k] = __uint_as_float(a[k]);
                v[k + 4] = __uint_as_float(b[k]);
            } else {
                typedef _Float16 h2 __attribute__((ext_vector_type(2)));
                const uint32_t w = a[k];  // by value: a bit cast of a vector's element takes element 0
                const h2 x = __builtin_bit_cast(h2, w);
                v[2 * k] = (float)x[0];
                v[2 * k + 1] = (float)x[1];
            }
        }
#pragma unroll
        for (int s = 0; s < kTerms<DT>; ++s)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int e0 = PAIR4 ? k : 2 * k, e1 = PAIR4 ? k + 4 : 2 * k + 1;
                const uint32_t b0 = __float_as_uint(v[e0]), b1 = __float_as_uint(v[e1]);
                t[s][k] = pack_hi(b0, b1);
                if (s + 1 < kTerms<DT>) {
                    v[e0] -= __uint_as_float(b0 & 0xffff0000u);
                    v[e1] -= __uint_as_float(b1 & 0xffff0000u);
                }
            }
    }
}
// The same and the sum of the eight elements.
template <int DT>
__device__ __forceinline__ void raw_terms_sum(const u32v4* raw, u32v4 (&t)[kTerms<DT>], float& sum) {
    raw_terms<DT, true>(raw, t);
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo = 0.0f, hi = 0.0f;  // from the smallest term up
#pragma unroll
        for (int s = kTerms<DT> - 1; s >= 0; --s) {
            const uint32_t w = t[s][k];
            lo += __uint_as_float(w << 16);
            hi += __uint_as_float(w & 0xffff0000u);
        }
        sum += lo + hi;
    }
}
template <int DT, bool PAIR4>
__device__ __forceinline__ void load_terms(const void* p, int64_t i, u32v4 (&t)[kTerms<DT>]) {
    const u32v4* q = (const u32v4*)((const char*)p + i * (DT == GPTQ_F32 ? 4 : 2));
    const u32v4 raw[2] = {q[0], DT == GPTQ_F32 ? q[1] : q[0]};
    raw_terms<DT, PAIR4>(raw, t);
}

// Eight values as kTerms operands, the last rounded to nearest even.
template <int DT>
__device__ __forceinline__ void weight_terms(float (&v)[8], u32v4 (&t)[kTerms<DT>]) {
#pragma unroll
    for (int s = 0; s + 1 < kTerms<DT>; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t b0 = __float_as_uint(v[2 * k]), b1 = __float_as_uint(v[2 * k + 1]);
            t[s][k] = pack_hi(b0, b1);
            v[2 * k] -= __uint_as_float(b0 & 0xffff0000u);
            v[2 * k + 1] -= __uint_as_float(b1 & 0xffff0000u);
        }
#pragma unroll
    for (int k = 0; k < 4; ++k) t[kTerms<DT> - 1][k] = round_bf16x2(v[2 * k], v[2 * k + 1]);
}

// (x & mask) | bits in one instruction, the mask in a scalar register and the bits in a vector one: with
// constants in sight the compiler takes an AND and an OR with literals instead, a third more of the
// unpacking.  The empty statements only hide the constants (no instruction is written by hand: the
// compiler has to see every write next to an MFMA to keep its distance from it).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    asm("" : "+s"(mask));
    asm("" : "+v"(bits));
    return (x & mask) | bits;
}
// Operand register n of a word of nibbles: codes (n, n + 4) as 16 + q.
template <int N>
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w) {
    const uint32_t x = N == 0 ? w << 3 : w >> (4 * N - 3);
    return and_or(x, 0x00780078u, 0x41804180u);
}
__device__ __forceinline__ u32v4 unpack_nibbles(uint32_t w) {
    return u32v4{nibble_pair<0>(w), nibble_pair<1>(w), nibble_pair<2>(w), nibble_pair<3>(w)};
}
constexpr uint32_t kMinus24 = 0xC1C0C1C0u;  // two of bf16's -24 = -(16 + 8)

// The nibbles of x at even or odd places, a byte each.  The empty statement hides the mask: seeing it, the
// compiler takes every byte out by a field extract of its own before it converts it.
__device__ __forceinline__ uint32_t nibble_bytes(uint32_t x, bool odd) {
    uint32_t y = (odd ? x >> 4 : x) & 0x0f0f0f0fu;
    asm("" : "+v"(y));
    return y;
}
// Codes in two registers' bytes times s, exact in bf16: (low half <- byte LO of y, high half <- byte HI).
template <int LO, int HI>
__device__ __forceinline__ uint32_t decode_pair(uint32_t y, float s0, float o0, float s1, float o1) {
    const float a = fmaf((float)(y >> (8 * LO) & 255u), s0, o0), b = fmaf((float)(y >> (8 * HI) & 255u), s1, o1);
    return pack_hi(__float_as_uint(a), __float_as_uint(b));
}

// Maximum and sum over the four lanes that share lane % 16.
__device__ __forceinline__ float quad_max(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// ---- the sequences of a call (gptq_batch), on the device ----

struct Batch {
    const int32_t* table;
    const int32_t* len;
    const int32_t* start;
    int seqs, width;
    int64_t rows;
};

// First and one-past-last row of sequence b, inside the call's rows whatever start holds.
__device__ __forceinline__ void seq_rows(const Batch& q, int b, int& r0, int& r1) {
    if (!q.start) {
        r0 = b;
        r1 = b + 1;
        return;
    }
    const int n = (int)q.rows;
    r0 = min(max(q.start[b], 0), n);
    r1 = min(max(q.start[b + 1], r0), n);
}

// The last b below n with at(b) <= x, of values that ascend, or -1: 64 of them a look.
template <class At>
__device__ __forceinline__ int last_at_most(int n, int x, At at) {
    const int lane = threadIdx.x & 63;
    int lo = 0;
    for (;;) {
        const int step = (n + 63) >> 6;
        const int before = __popcll(__ballot(lane * step < n && at(lo + min(lane * step, n - 1)) <= x)) - 1;
        if (before < 0) return -1;  // not behind the first look, where starts ascend
        lo += before * step;
        if (step == 1) return lo;
        n = min(step, n - before * step);
    }
}

// Sequence of a row (the same in every lane), or -1 behind the last or before the first.
__device__ __forceinline__ int seq_of_row(const Batch& q, int row) {
    if (!q.start) return row;
    const int b = last_at_most(q.seqs, row, [&](int i) { return q.start[i]; });
    return b >= 0 && q.start[b + 1] > row ? b : -1;
}

}  // namespace gptq
