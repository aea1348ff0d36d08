// rotary.hip -- rotary positions on gfx950.
//
// Pair i of the first `part` channels of a head is turned by the angle position x freq[i] and multiplied by
// `factor`: (a, b) -> (a cos - b sin, b cos + a sin).  Pairs are channels (i, i + part / 2) or (2 i, 2 i + 1);
// channels from `part` on stay.  The turn's transpose (backward) takes sin from the other side.
//
// Angles are f64: the turn count position freq / 2 pi is taken as a sum of two doubles, so that its fraction, which goes
// to sincospif, is off by less than f32 shows at every position (rounded to one double it is 3.9e-7 off near 2^31, f32's
// own 0.9e-7).  All heads of a row share them, so a workgroup makes the cosines and sines
// of its rows once, in LDS, and then walks over heads with 16-byte vectors.  Bound by memory: 20000 rows of 40 heads of
// 128 in f16, half of the channels turned, take 83 us, 4.9 TB/s, a copy's rate.
#include "check.hpp"
#include "codes16.hpp"
#include "common.hpp"

namespace gptq {

constexpr int kRotaryThreads = 256, kRotaryPairs = 1024, kRotaryTensors = 4;

struct RotaryArgs {
    gptq_rotated t[kRotaryTensors];
    int count, heads;  // heads of all tensors
    int rows, dim, part;
    const int32_t* position;
    const double* freq;
    float factor, sign;
    int block;  // rows of a workgroup
};

// position freq / 2 pi less a whole number, within 1/2 and a rounding: each product with what it leaves.
__device__ __forceinline__ double turn_part(double position, double freq) {
#pragma clang fp contract(off)  // a product fused into the difference would count its rest twice
    constexpr double k = 0x1.45f306dc9c883p-3, k_rest = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
    const double angle = position * freq, angle_rest = fma(position, freq, -angle);
    const double turns = angle * k, rest = fma(angle, k, -turns) + fma(angle, k_rest, angle_rest * k);
    return turns - rint(turns) + rest;
}

// One element or a vector of E of them as floats.
template <int DT, int E>
__device__ __forceinline__ void rot_load(const void* p, int64_t i, float (&v)[E]) {
    if constexpr (E == 1) {
        v[0] = load_one<DT>(p, i);
    } else if constexpr (E == 4) {
        const f32v4 x = *(const f32v4*)((const float*)p + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = x[k];
    } else {
        load_eight<DT>(p, i, v);
    }
}
template <int DT, int E>
__device__ __forceinline__ void rot_store(void* p, int64_t i, const float (&v)[E]) {
    if constexpr (E == 1)
        store_one<DT>(p, i, v[0]);
    else if constexpr (E == 4)
        *(f32v4*)((float*)p + i) = f32v4{v[0], v[1], v[2], v[3]};
    else
        store_eight<DT>(p, i, v);
}

// E elements a vector: 16 bytes, or 1 where sizes or addresses do not allow that.  A unit is a vector of each
// half of the turned channels, or (NEXT: neighbours are pairs) two vectors in a row; behind the units of a
// head follow its unturned vectors.
template <int DT, int E, bool NEXT>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(RotaryArgs a) {
    __shared__ float cs[2 * kRotaryPairs];
    const int row0 = blockIdx.x * a.block, n = min(a.block, a.rows - row0);
    const int half = a.part >> 1;
    for (int u = threadIdx.x; u < n * half; u += kRotaryThreads) {
        const int r = u / half, i = u - r * half;
        float s, c;
        sincospif((float)(2.0 * turn_part((double)a.position[row0 + r], a.freq[i])), &s, &c);
        cs[2 * u] = c * a.factor;
        cs[2 * u + 1] = s * a.sign;
    }
    __syncthreads();
    // A thread has one unit of every `slots`-th head, so that a row's cosines and sines stay in registers.
    const int turned = half / E, units = turned + (a.dim - a.part) / E;
    const int wide = min(units, kRotaryThreads), slots = kRotaryThreads / wide;
    const int slot = threadIdx.x / wide, first = slot + blockIdx.y * slots, step = slots * gridDim.y;
    if (slot >= slots) return;
    for (int u = threadIdx.x - slot * wide; u < units; u += wide) {
        const bool turns = u < turned;
        const int d0 = !turns ? a.part + (u - turned) * E : NEXT ? 2 * u * E : u * E, d1 = NEXT ? d0 + E : d0 + half;
        for (int r = 0; r < n; ++r) {
            float c[E], s[E];
            if (turns) {
                const float* m = cs + 2 * (r * half + u * E);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    c[e] = m[2 * e];
                    s[e] = m[2 * e + 1];
                }
            }
            int head = first;
            for (int k = 0; k < a.count; ++k) {
                const gptq_rotated& t = a.t[k];
                const int64_t from = (int64_t)(row0 + r) * t.ldx, to = (int64_t)(row0 + r) * t.ldy;
                for (; head < t.heads; head += step) {
                    const int64_t x = from + head * t.ldxh, o = to + head * t.ldyh;
                    float p[E], q[E];
                    if (!turns) {
                        if (t.X == t.Y) continue;
                        rot_load<DT, E>(t.X, x + d0, p);
                        rot_store<DT, E>(t.Y, o + d0, p);
                        continue;
                    }
                    rot_load<DT, E>(t.X, x + d0, p);
                    rot_load<DT, E>(t.X, x + d1, q);
                    float y[E], z[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        // Pair e of the unit: its channels are elements 2 e and 2 e + 1 of the two vectors, or e of each.
                        const int e0 = 2 * e, e1 = 2 * e + 1;
                        const float v0 = !NEXT ? p[e] : e0 < E ? p[e0 % E] : q[e0 % E], v1 = !NEXT ? q[e] : e1 < E ? p[e1 % E] : q[e1 % E];
                        const float o0 = fmaf(v0, c[e], -v1 * s[e]), o1 = fmaf(v1, c[e], v0 * s[e]);
                        if constexpr (!NEXT) {
                            y[e] = o0;
                            z[e] = o1;
                        } else {
                            (e0 < E ? y : z)[e0 % E] = o0;
                            (e1 < E ? y : z)[e1 % E] = o1;
                        }
                    }
                    rot_store<DT, E>(t.Y, o + d0, y);
                    rot_store<DT, E>(t.Y, o + d1, z);
                }
                head -= t.heads;
            }
        }
    }
}

typedef void (*RotaryKernel)(RotaryArgs);
template <int DT>
static RotaryKernel rotary_pick(bool vec, bool next) {
    constexpr int E = DT == GPTQ_F32 ? 4 : 8;
    if (vec) return next ? rotary_kernel<DT, E, true> : rotary_kernel<DT, E, false>;
    return next ? rotary_kernel<DT, 1, true> : rotary_kernel<DT, 1, false>;
}

// A tensor's rows as memory: whole rows where its heads lie side by side in them, else the heads of each row
// (or, with rows inside heads, the rows of each head) one by one would be needed: its whole range.
static RowSet rotated_rows(const void* p, int64_t ld, int64_t ldh, int64_t rows, int64_t heads, int dim, int es) {
    if (heads == 1 || ldh == dim) return RowSet{p, ld * es, rows, heads * dim * es};
    const int64_t all = ((rows - 1) * ld + (heads - 1) * ldh + dim) * es;
    return RowSet{p, all, 1, all};
}
// Rows and heads at strides that give no element twice.
static bool rotated_ok(int64_t ld, int64_t ldh, int64_t rows, int64_t heads, int dim) {
    const int64_t most = (int64_t)1 << 36;
    return ld >= dim && ldh >= dim && ld <= most && ldh <= most && (ld >= (heads - 1) * ldh + dim || ldh >= (rows - 1) * ld + dim);
}

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_rotary(const gptq_rotated* tensors, int32_t count, int dtype, int64_t rows, int32_t dim, int32_t part,
                           int layout, const int32_t* position, const double* freq, float factor, int backward, void* stream) {
    const int es = dtype_size(dtype);
    if (!es || !tensors || count < 1 || count > kRotaryTensors || rows < 0 || rows > (1 << 23) || dim < 1 || dim > 2 * kRotaryPairs ||
        part < 2 || part > dim || part % 2 || (layout != GPTQ_ROTARY_HALF && layout != GPTQ_ROTARY_NEXT) || !(factor - factor == 0.0f))
        return GPTQ_EINVAL;
    RotaryArgs a{};
    for (int i = 0; i < count; ++i) {
        if (tensors[i].heads < 1 || tensors[i].heads > 65535) return GPTQ_EINVAL;
        a.t[i] = tensors[i];
        a.heads += tensors[i].heads;
    }
    if ((int64_t)a.heads * dim > (1 << 26)) return GPTQ_EINVAL;  // a workgroup's elements stay below 2^31
    if (rows == 0) return GPTQ_OK;
    if (!position || !freq || ((uintptr_t)position & 3u) || ((uintptr_t)freq & 7u)) return GPTQ_EINVAL;
    const int E = 16 / es;
    bool vec = (part / 2) % E == 0 && (dim - part) % E == 0;
    for (int i = 0; i < count; ++i) {
        const gptq_rotated& t = tensors[i];
        if (!t.X || !t.Y || !rotated_ok(t.ldx, t.ldxh, rows, t.heads, dim) || !rotated_ok(t.ldy, t.ldyh, rows, t.heads, dim) ||
            ((uintptr_t)t.X | (uintptr_t)t.Y) % (unsigned)es)
            return GPTQ_EINVAL;
        vec = vec && al16(t.X) && al16(t.Y) && (t.ldx | t.ldxh | t.ldy | t.ldyh) % E == 0;
        // In place, a pair is read and written by one thread.
        const bool in_place = t.X == t.Y && (rows == 1 || t.ldx == t.ldy) && (t.heads == 1 || t.ldxh == t.ldyh);
        const RowSet y = rotated_rows(t.Y, t.ldy, t.ldyh, rows, t.heads, dim, es);
        if (rows_meet(y, RowSet{position, 4 * rows, 1, 4 * rows}) || rows_meet(y, RowSet{freq, 4 * part, 1, 4 * part})) return GPTQ_EINVAL;
        for (int k = 0; k < count; ++k) {
            const gptq_rotated& o = tensors[k];
            if (!(k == i && in_place) && rows_meet(y, rotated_rows(o.X, o.ldx, o.ldxh, rows, o.heads, dim, es))) return GPTQ_EINVAL;
            if (k != i && rows_meet(y, rotated_rows(o.Y, o.ldy, o.ldyh, rows, o.heads, dim, es))) return GPTQ_EINVAL;
        }
    }
    CheckScope check;
    check_buffer(position, 4 * (size_t)rows, "position");
    check_buffer(freq, 4 * (size_t)part, "freq");
    for (int i = 0; i < count; ++i) {
        const gptq_rotated& t = tensors[i];
        check_buffer(t.X, (size_t)((rows - 1) * t.ldx + (t.heads - 1) * t.ldxh + dim) * (size_t)es, "X");
        check_buffer(t.Y, (size_t)((rows - 1) * t.ldy + (t.heads - 1) * t.ldyh + dim) * (size_t)es, "Y");
    }
    a.count = count;
    a.rows = (int)rows;
    a.dim = dim;
    a.part = part;
    a.position = position;
    a.freq = freq;
    a.factor = factor;
    a.sign = backward ? -factor : factor;
    // Rows of a workgroup: what LDS holds of their angles, and not so many that CUs are left without.  (20000 rows of 40
    // heads, half of 128 channels turned, f16: two rows 83 us, four 87, eight 103.)
    int64_t block = kRotaryPairs / (part / 2), share = rows / (4 * kCUs);
    if (share < 1) share = 1;
    if (block > share) block = share;
    if (block > 2) block = 2;
    a.block = (int)block;
    const int64_t units = (part / 2 + dim - part) / (vec ? E : 1), slots = units < kRotaryThreads ? kRotaryThreads / units : 1;
    int64_t slices = (a.heads + slots - 1) / slots;
    const int64_t wg = (rows + block - 1) / block;
    const int64_t room = (4 * kCUs + wg - 1) / wg;  // workgroups that share a row's heads, where rows are few
    if (slices > room) slices = room;
    hipStream_t st = (hipStream_t)stream;
    const RotaryKernel k = dtype == GPTQ_F32    ? rotary_pick<GPTQ_F32>(vec, layout == GPTQ_ROTARY_NEXT)
                           : dtype == GPTQ_BF16 ? rotary_pick<GPTQ_BF16>(vec, layout == GPTQ_ROTARY_NEXT)
                                                : rotary_pick<GPTQ_F16>(vec, layout == GPTQ_ROTARY_NEXT);
    auto span = [&](int i, bool write) {
        const gptq_rotated& t = tensors[i < count ? i : 0];
        const int64_t ld = write ? t.ldy : t.ldx, ldh = write ? t.ldyh : t.ldxh;
        const int64_t wide = ld >= ldh ? (t.heads - 1) * ldh + dim : dim;
        Span s = rd(write ? t.Y : t.X, ld >= ldh ? ld : ldh, i < count ? (ld >= ldh ? rows : t.heads) : 0, ld >= ldh ? wide : (rows - 1) * ld + dim, es);
        s.write = write;
        return s;
    };
    {
        ProfScope ps(FAM_ATTENTION, st, 0.0, 2.0 * (double)rows * a.heads * dim * es);
        GPTQ_LAUNCH(st, "rotary", (k<<<dim3((unsigned)wg, (unsigned)slices), kRotaryThreads, 0, st>>>(a)), rd(position, rows, 1, rows),
                    rd(freq, part / 2, 1, part / 2, 8), span(0, false), span(1, false), span(2, false), span(3, false),
                    span(0, true), span(1, true), span(2, true), span(3, true));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}
