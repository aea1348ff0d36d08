// dense16.hpp -- products of many tokens whose operands are both laid out in f16, and what makes them: the gated
// block and the gradients (gated.hip, backward.hip).
//
// W = W' 2^p, p a power of two of each of the sweep's rows, W' its codes times what is left of the scales, rounded to
// f16's 11 bits; X = X' 2^e, e of each token, exact in f16 for bf16 and f16 activations but for values below
// 2^-28 of their token's largest, which are rounded to that.  So bf16 loses nothing to its 8 bits on the way
// (weights rounded to them give sums 0.0017 off, as much as the output's own rounding), and the matrix
// units run at the same rate.
//
// f16 results have 11 bits themselves, and behind two products and an activation weights of 11 bits put the block
// 3.6e-4 off and its gradient 4.4e-4, where one rounding is 2.1e-4.  There the block's W' is two terms, 22 bits, and so
// are the gradients of its sums, kTileK columns of each in turn, each with the same tile of the other operand: twice the
// products (twice the time), block and rounding alike 2.1e-4, the gradient 2.9e-4, what the last product's weights of 11
// bits leave.
//
// dense16_kernel is linear_dense.hpp's tiled product with other epilogues:
//   DENSE_PLAIN  Y = z                       (W turned: the gradient of X)
//   DENSE_GATED  Y = act(a + bias) (b + bias2)
//   DENSE_GRAD   the gradients of a and b, as the next product's X'
//   DENSE_LAST   that product: DENSE_PLAIN, of an X' in two terms in f16.
// For the last two W' holds both matrices in turns of 16 rows (linear_codes.hpp, sums_of).
#pragma once
#include "linear_dense.hpp"

namespace gptq {

enum { DENSE_PLAIN = 0, DENSE_GATED = 1, DENSE_GRAD = 2, DENSE_LAST = 3 };
constexpr bool dense_plain(int mode) { return mode == DENSE_PLAIN || mode == DENSE_LAST; }
// Terms of the block's W', and of the gradients of its sums.
constexpr int block_terms(int type) { return type == GPTQ_F16 ? 2 : 1; }
// Column c of such an operand's first term.
__device__ __forceinline__ int two_term_column(int c) { return c / kTileK * (2 * kTileK) + c % kTileK; }

// What bounds the gradients of a and b, whatever the weights are (grad_exponent): the rows' largest, in a slot of
// each row's number modulo kSlots.
constexpr int kSlots = 64;
struct GradBound {
    float sums[kSlots], bias[kSlots];
};

struct Dense16 {
    const uint16_t* X;    // X' [t, ldx]
    int ldx, t;
    const uint16_t* W;    // W' [whole tiles of sums, ldw]
    int ldw;
    const float* power;   // 2^p of each row of W', or NULL: 1 (W turned)
    const float* token;   // 2^e of each token
    int rows, act;        // columns of Y (one matrix's rows)
    const float* bias;
    const float* bias2;
    void* Y;
    int64_t ldy;
    int tiles_r, tiles, whole, splits;
    float* part;
    // DENSE_GRAD: the gradient of Y, the result [t, 2 side], one or two terms, and the 2^e of its tokens.
    const void* dY;
    int64_t ldd;
    uint16_t* D;
    int side;
    const float* grad_token;
};

// |dy| act'(a) |b| 2^p and |dy| |act(a)| 2^p, the gradients before a token's power is taken out, are at most
// top_dy 1.13 (top_x sums + bias), sums = the largest 2^p' sum |w| (p' the power of a row of one matrix, w
// the same row of the other), bias the largest 2^p' |bias|; no activation has a slope over 1.13 or a magnitude over its
// argument's, nor one over 0.28 of negative arguments: a gate that its bias shuts counts with that (with |bias|, gates
// shut by -1e30 flushed every other's gradient to zero).  The exponent that brings this to 2^15, below f16's 65504.  Actual
// gradients lie some 2^10 below; f16 has another 2^24 under those before it rounds them harder.
__device__ __forceinline__ int grad_exponent(float top_dy, float top_x, float sums, float bias) {
    const float x = top_dy * fmaf(top_x, sums, bias) * 1.13f;
    if (!(x > 0.0f)) return 0;
    return x < INFINITY ? min(max(ilogbf(x) - 14, -126), 126) : 126;
}

// Eight columns of Y from r on: their rows' powers and biases in the two matrices.  Loaded once a lane.
struct Columns {
    int r;
    float p[8], q[8], a[8], b[8];
    __device__ __forceinline__ void load(const Dense16& d, int first) {
        r = first;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            const int rr = min(r + v, d.rows - 1);
            const float* two = d.power + (rr >> 4) * 32 + (rr & 15);
            p[v] = two[0];
            q[v] = two[16];
            a[v] = d.bias ? d.bias[rr] : 0.0f;
            b[v] = d.bias2 ? d.bias2[rr] : 0.0f;
        }
    }
};
// Those of a token: sums a and b of the two matrices.
template <int DT, int MODE>
__device__ __forceinline__ void finish_eight(const Dense16& d, int tok, const Columns& k, float (&a)[8], float (&b)[8], bool aligned) {
    const float two = d.token[tok];
    const int r = k.r;
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        a[v] = fmaf(a[v] * k.p[v], two, k.a[v]);
        b[v] = fmaf(b[v] * k.q[v], two, k.b[v]);
    }
    if constexpr (MODE == DENSE_GATED) {
        gate_all<true>(a, b, d.act);
        if (aligned && r + 8 <= d.rows) {
            store_eight<DT>(d.Y, (int64_t)tok * d.ldy + r, a);
        } else {
#pragma unroll
            for (int v = 0; v < 8; ++v)
                if (r + v < d.rows) store_one<DT>(d.Y, (int64_t)tok * d.ldy + r + v, a[v]);
        }
    } else {
        float dy[8];
        if (aligned && r + 8 <= d.rows) {
            load_eight<DT>(d.dY, (int64_t)tok * d.ldd + r, dy);
        } else {
#pragma unroll
            for (int v = 0; v < 8; ++v) dy[v] = r + v < d.rows ? load_one<DT>(d.dY, (int64_t)tok * d.ldd + r + v) : 0.0f;
        }
        const float less = 1.0f / d.grad_token[tok];  // exact: a power of two
        gated_grads<true>(a, b, dy, d.act);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            // Columns behind the last are zeros, whatever the sums of rows that are not there hold.
            a[v] = r + v < d.rows ? a[v] * less * k.p[v] : 0.0f;
            b[v] = r + v < d.rows ? b[v] * less * k.q[v] : 0.0f;
        }
        if (r < d.side) {
            if constexpr (block_terms(DT) == 2) {
                uint16_t* o = d.D + (int64_t)tok * (4 * d.side);
                const int i = two_term_column(r), j = two_term_column(d.side + r);
                store_eight<GPTQ_F16>(o, i, a);
                store_eight<GPTQ_F16>(o, j, b);
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    a[v] = what_f16_leaves(a[v]);
                    b[v] = what_f16_leaves(b[v]);
                }
                store_eight<GPTQ_F16>(o, i + kTileK, a);
                store_eight<GPTQ_F16>(o, j + kTileK, b);
            } else {
                uint16_t* o = d.D + (int64_t)tok * (2 * d.side) + r;
                store_eight<GPTQ_F16>(o, 0, a);
                store_eight<GPTQ_F16>(o, d.side, b);
            }
        }
    }
}

template <int DT, int MODE>
__global__ __launch_bounds__(kDenseWaves * 64) void dense16_kernel(Dense16 d) {
    __shared__ __attribute__((aligned(16))) uint16_t xs0[kTileT * kTileK];
    __shared__ __attribute__((aligned(16))) uint16_t ws0[kTileR * kTileK];
    __shared__ __attribute__((aligned(16))) uint16_t xs1[kTileT * kTileK];
    __shared__ __attribute__((aligned(16))) uint16_t ws1[kTileR * kTileK];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int wt = wave >> 2, wr = wave & 3;
    int tile = blockIdx.x, split = 0;
    const bool cut = tile >= d.whole;
    if (cut) {
        split = (tile - d.whole) % d.splits;
        tile = d.whole + (tile - d.whole) / d.splits;
    }
    const int tok0 = tile / d.tiles_r * kTileT, row0 = tile % d.tiles_r * kTileR;
    constexpr int XS = !dense_plain(MODE) && block_terms(DT) == 2, WS = MODE == DENSE_LAST && block_terms(DT) == 2;
    const int all = (XS ? d.ldw : d.ldx) / kTileK;
    const int first = cut ? (int)((int64_t)all * split / d.splits) : 0;
    const int steps = cut ? (int)((int64_t)all * (split + 1) / d.splits) : all;
    f32v4 acc[4][8];
    dense_sums<GPTQ_F16, XS, WS>(d.X, d.ldx, d.t, tok0, d.W, d.ldw, row0, d.ldx, first, steps, all, xs0, ws0, xs1, ws1, acc);
    if (cut) {
        float* mine = d.part + ((int64_t)(tile - d.whole) * d.splits + split) * (kTileT * kTileR);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *(f32v4*)(mine + ((i * 8 + j) * (kDenseWaves * 64) + threadIdx.x) * 4) = acc[i][j];
        return;
    }
    // By way of LDS, 64 tokens x 64 sums of a wave at a time: four lanes then hold a token's.
    float* buf = (float*)(wave < 2 ? xs0 : wave < 4 ? ws0 : wave < 6 ? xs1 : ws1) + (wave & 1) * 4096;
    const int v0 = row0 + wr * 64;  // the wave's first column of sums
    Columns own;
    if constexpr (!dense_plain(MODE)) own.load(d, (v0 >> 1) + (lane & 3) * 8);
    const void* out = MODE == DENSE_GRAD ? d.dY : d.Y;
    const int64_t ld = MODE == DENSE_GRAD ? d.ldd : d.ldy;
    const bool aligned = ld % 8 == 0 && ((uintptr_t)out & 15u) == 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(f32v4*)(buf + (j * 16 + c) * 64 + (((i * 4 + h) ^ c) << 2)) = acc[i][half * 4 + j];
        __builtin_amdgcn_wave_barrier();
        auto four = [&](int tt, int col) { return *(const f32v4*)(buf + tt * 64 + (((col >> 2) ^ (tt & 15)) << 2)); };
        if constexpr (dense_plain(MODE)) {
            if (!aligned) {  // a column a lane: neighbours store side by side
                const int r = v0 + lane;
#pragma unroll 1
                for (int tt = 0; tt < 64; ++tt) {
                    const int tok = tok0 + wt * 128 + half * 64 + tt;
                    if (tok >= d.t) break;
                    const float z = buf[tt * 64 + (((lane >> 2) ^ (tt & 15)) << 2) + (lane & 3)] * d.token[tok];
                    if (r < d.rows) store_one<DT>(d.Y, (int64_t)tok * d.ldy + r, z);
                }
                __builtin_amdgcn_wave_barrier();
                continue;
            }
        }
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            const int tt = q * 16 + (lane >> 2), tok = tok0 + wt * 128 + half * 64 + tt, s = lane & 3;
            if constexpr (dense_plain(MODE)) {
                const int r = v0 + s * 16;
                float z[16];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const f32v4 y = four(tt, s * 16 + 4 * u);
#pragma unroll
                    for (int v = 0; v < 4; ++v) z[4 * u + v] = y[v];
                }
                if (tok >= d.t) continue;
                const float two = d.token[tok];
#pragma unroll
                for (int v = 0; v < 16; ++v) z[v] *= two;
                const int64_t yo = (int64_t)tok * d.ldy + r;
                if (r + 16 <= d.rows) {
                    store_eight<DT>(d.Y, yo, z);
                    store_eight<DT>(d.Y, yo + 8, z + 8);
                } else {
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        if (r + v < d.rows) store_one<DT>(d.Y, yo + v, z[v]);
                }
            } else {
                const int col = (s >> 1) * 32 + 8 * (s & 1);  // of the sums; the second matrix's are 16 on
                float a[8], b[8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const f32v4 y = four(tt, col + 4 * u), z = four(tt, col + 16 + 4 * u);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        a[4 * u + v] = y[v];
                        b[4 * u + v] = z[v];
                    }
                }
                if (tok >= d.t) continue;
                finish_eight<DT, MODE>(d, tok, own, a, b, aligned);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// The sums of a cut tile's pieces, in their order, and the epilogue.  A thread has four neighbouring columns of
// sums of a token, in the order the pieces were written; of two matrices, those of both, and the next four from
// the lane beside it.
template <int DT, int MODE>
__global__ __launch_bounds__(256) void dense16_join_kernel(Dense16 d) {
    constexpr int T = kDenseWaves * 64;
    const int tile = d.whole + blockIdx.y;
    const int u = blockIdx.x * 256 + threadIdx.x;
    const float* part = d.part + (int64_t)blockIdx.y * d.splits * (kTileT * kTileR);
    auto sum = [&](int at) {
        const float* p = part + 4 * at;
        f32v4 z = *(const f32v4*)p;
        for (int s = 1; s < d.splits; ++s) z += *(const f32v4*)(p + (int64_t)s * (kTileT * kTileR));
        return z;
    };
    if constexpr (dense_plain(MODE)) {
        const int thread = u % T, i = u / T >> 3, j = u / T & 7, lane = thread & 63, wave = thread >> 6;
        const int r = tile % d.tiles_r * kTileR + (wave & 3) * 64 + i * 16 + 4 * (lane >> 4);
        const int tok = tile / d.tiles_r * kTileT + (wave >> 2) * 128 + j * 16 + (lane & 15);
        if (tok >= d.t || r >= d.rows) return;
        const f32v4 z = sum(u);
        const float two = d.token[tok];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (r + v < d.rows) store_one<DT>(d.Y, (int64_t)tok * d.ldy + r + v, z[v] * two);
    } else {
        // u counts (i / 2, j, wave, pair of quarters, token): eight columns of one matrix's rows.
        const int tl = u & 15, hh = u >> 4 & 1, wave = u >> 5 & 7, j = u >> 8 & 7, i2 = u >> 11 & 1;
        const int r = ((tile % d.tiles_r * kTileR + (wave & 3) * 64) >> 1) + i2 * 16 + 8 * hh;
        const int tok = tile / d.tiles_r * kTileT + (wave >> 2) * 128 + j * 16 + tl;
        if (tok >= d.t || r >= (MODE == DENSE_GRAD ? d.side : d.rows)) return;
        float a[8], b[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int at = (2 * i2 * 8 + j) * T + wave * 64 + (2 * hh + k) * 16 + tl;
            const f32v4 y = sum(at), z = sum(at + 8 * T);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                a[4 * k + v] = y[v];
                b[4 * k + v] = z[v];
            }
        }
        const void* out = MODE == DENSE_GRAD ? d.dY : d.Y;
        const int64_t ld = MODE == DENSE_GRAD ? d.ldd : d.ldy;
        Columns own;
        own.load(d, r);
        finish_eight<DT, MODE>(d, tok, own, a, b, ld % 8 == 0 && ((uintptr_t)out & 15u) == 0);
    }
}

// ---- what the product reads ----

// One workgroup per token: X' [t, ldx] and 2^e, times 2^p of each column (power, or NULL).  top: the largest
// magnitudes (or NULL).  X' reaches 2^15 at most.  ldx is n rounded up; zeros behind n.  Without H the token's
// power is that of the gated block's gradients, from dY in X's place.
struct Halve {
    const void* X;
    int64_t ld;
    int n;
    const float* power;
    uint16_t* H;
    int ldh;
    float* token;
    float* top;              // of X's; read where H is NULL
    const GradBound* bound;  // read where H is NULL
};
template <int DT>
__global__ __launch_bounds__(256) void halve_kernel(Halve a) {
    constexpr int HELD = 4;  // vectors a thread keeps between its two looks at them: rows of up to 8192
    __shared__ float part[4];
    const int tok = blockIdx.x;
    const char* x = (const char*)a.X + (int64_t)tok * a.ld * 2;
    // 16-byte loads, where a row starts and ends on them.
    const bool vec = a.n % 8 == 0 && ((uintptr_t)x & 15u) == 0;
    auto load = [&](int u, float (&v)[8]) {
        if (vec && 8 * u < a.n) {
            load_eight<DT>(x, 8 * u, v);
            if (a.power) {
                const f32v4 p = *(const f32v4*)(a.power + 8 * u), q = *(const f32v4*)(a.power + 8 * u + 4);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= k < 4 ? p[k & 3] : q[k & 3];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 8 * u + k < a.n ? load_one<DT>(x, 8 * u + k) * (a.power ? a.power[8 * u + k] : 1.0f) : 0.0f;
        }
    };
    float most = 0.0f, kept[HELD][8];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        load(threadIdx.x + i * 256, kept[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) most = fmaxf(most, fabsf(kept[i][k]));
    }
    for (int u = threadIdx.x + HELD * 256; u < (a.n + 7) / 8; u += 256) {
        float v[8];
        load(u, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) most = fmaxf(most, fabsf(v[k]));
    }
#pragma unroll
    for (int k = 1; k < 64; k *= 2) most = fmaxf(most, __shfl_xor(most, k));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = most;
    __syncthreads();
    most = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    if (!a.H) {
        if (threadIdx.x >= 64) return;
        float sums = a.bound->sums[threadIdx.x], bias = a.bound->bias[threadIdx.x];
#pragma unroll
        for (int k = 1; k < 64; k *= 2) {
            sums = fmaxf(sums, __shfl_xor(sums, k));
            bias = fmaxf(bias, __shfl_xor(bias, k));
        }
        if (threadIdx.x == 0) a.token[tok] = ldexpf(1.0f, grad_exponent(most, a.top[tok], sums, bias));
        return;
    }
    if (a.top && threadIdx.x == 0) a.top[tok] = most;
    int e = 0;
    if (most > 0.0f && most < INFINITY) e = min(max(ilogbf(most) - 14, -126), 126);
    const float less = ldexpf(1.0f, -e);
    if (threadIdx.x == 0) a.token[tok] = ldexpf(1.0f, e);
    uint16_t* to = a.H + (int64_t)tok * a.ldh;
    auto store = [&](int u, float (&v)[8]) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= less;
        store_eight<GPTQ_F16>(to, 8 * u, v);
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        if (threadIdx.x + i * 256 < a.ldh / 8) store(threadIdx.x + i * 256, kept[i]);
    for (int u = threadIdx.x + HELD * 256; u < a.ldh / 8; u += 256) {
        float v[8];
        load(u, v);
        store(u, v);
    }
}

// The two matrices' row r, decoded in turns of 16 rows (ldx columns, one term or two), with their powers and (bound
// given) what bounds their gradients, of the sums and of the biases.  One workgroup per row.
template <int BITS, bool TWO>
__global__ __launch_bounds__(256) void decode_two_kernel(LinArgs a, uint16_t* W, float* power, int ldx, f32v2* bound) {
    const int64_t ldw = (int64_t)ldx * (TWO ? 2 : 1);
    __shared__ float part[2][4];
    const int64_t row = blockIdx.x, v = (row >> 4) * 32 + (row & 15);
    const float* sp[2] = {a.scale + row * a.G, a.scale2 + row * a.G};
    const uint8_t* cp[2] = {a.codes + row * a.G * (4 * BITS), a.codes2 + row * a.G * (4 * BITS)};
    float two[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int e = row_exponent(sp[m], a.G, part[m]);
        two[m] = ldexpf(1.0f, e);
        if (threadIdx.x == 0) power[v + 16 * m] = two[m];
        decode_row<GPTQ_F16, BITS, TWO>(cp[m], sp[m], a.G, ldexpf(1.0f, -e), W + (v + 16 * m) * ldw, ldx);
    }
    if (!bound) return;
    __syncthreads();  // `part` again
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        // sum |w| is at most 32 top |s| a group, top the largest level.
        float sum = 0.0f;
        for (int g = threadIdx.x; g < a.G; g += 256) sum += fabsf(sp[m][g]);
#pragma unroll
        for (int k = 1; k < 64; k *= 2) sum += __shfl_xor(sum, k);
        if ((threadIdx.x & 63) == 0) part[m][threadIdx.x >> 6] = sum;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float x = 0.0f, b = 0.0f;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float* bp = m ? a.bias2 : a.bias;
            x = fmaxf(x, (part[m][0] + part[m][1] + part[m][2] + part[m][3]) * (32.0f * (BITS == 4 ? 8.0f : 1.5f)) * two[1 - m]);
            if (!bp) continue;
            const float v = bp[row];
            b = fmaxf(b, (m == 0 && a.act != GPTQ_ACT_NONE && v < 0.0f ? fminf(-v, 0.28f) : fabsf(v)) * two[1 - m]);
        }
        bound[row] = f32v2{x, b};
    }
}
// Slot blockIdx.x of the rows' bounds, kSlots workgroups.  A launch of its own: every row's atomic on the slots
// made decode_two_kernel of two 17408 x 5120 140 us long; without them it takes 97 (two terms 174), and this kernel 5.
__global__ __launch_bounds__(256) static void bound_kernel(const f32v2* row_bound, int rows, GradBound* bound) {
    __shared__ float part[2][4];
    float x = 0.0f, b = 0.0f;
    for (int r = threadIdx.x * kSlots + blockIdx.x; r < rows; r += 256 * kSlots) {
        const f32v2 v = row_bound[r];
        x = fmaxf(x, v[0]);
        b = fmaxf(b, v[1]);
    }
#pragma unroll
    for (int k = 1; k < 64; k *= 2) {
        x = fmaxf(x, __shfl_xor(x, k));
        b = fmaxf(b, __shfl_xor(b, k));
    }
    if ((threadIdx.x & 63) == 0) {
        part[0][threadIdx.x >> 6] = x;
        part[1][threadIdx.x >> 6] = b;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        const float* v = part[threadIdx.x];
        (threadIdx.x ? bound->bias : bound->sums)[blockIdx.x] = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
    }
}

// 2^p of each row of a matrix: one workgroup a row.
__global__ __launch_bounds__(256) static void row_power_kernel(const float* scale, int G, float* power) {
    __shared__ float part[4];
    const int e = row_exponent(scale + (int64_t)blockIdx.x * G, G, part);
    if (threadIdx.x == 0) power[blockIdx.x] = ldexpf(1.0f, e);
}

// W' turned: T [n, ldt], T[j][m side + r] = W'_m[r][j], zeros for r from `rows` to side - 1 (side a multiple of 64).
// A wave takes 64 rows and 64 columns: a lane the 8 x 8 block of rows 8 (l % 8) .. and columns 8 (l / 8) .., a word
// of codes a row, and stores 16 bytes a column, eight lanes 128 bytes side by side.
struct Turn {
    const uint8_t* codes[2];
    const float* scale[2];
    const float* power;  // row r's: of one matrix at r, of two (`turns`) at (r / 16) 32 + 16 m + r % 16
    bool turns;
    int rows, n, side, ldt;
    uint16_t* T;
};
template <int BITS>
__global__ __launch_bounds__(256) void turn_kernel(Turn a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = blockIdx.z;
    const int r0 = blockIdx.y * 64 + 8 * (lane & 7), j0 = blockIdx.x * 256 + wave * 64 + 8 * (lane >> 3);
    if (j0 >= a.n) return;
    const int64_t G = a.n / 32;
    const uint8_t* codes = m ? a.codes[1] : a.codes[0];
    const float* scale = m ? a.scale[1] : a.scale[0];
    uint32_t w[8];
    float s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t r = min(r0 + k, a.rows - 1), at = (r * a.n + j0) / 8;
        w[k] = BITS == 4 ? ((const uint32_t*)codes)[at] : (uint32_t)((const uint16_t*)codes)[at];
        const float two = a.power[a.turns ? (r >> 4) * 32 + 16 * m + (r & 15) : r];
        s[k] = scale[r * G + (j0 >> 5)] * (1.0f / two);  // exact: a power of two
    }
    uint16_t* to = a.T + (int64_t)j0 * a.ldt + (int64_t)m * a.side + r0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u32v4 o;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x = r0 + 2 * k < a.rows ? level<BITS>(w[2 * k] >> (BITS * i)) * s[2 * k] : 0.0f;
            const float y = r0 + 2 * k + 1 < a.rows ? level<BITS>(w[2 * k + 1] >> (BITS * i)) * s[2 * k + 1] : 0.0f;
            o[k] = pack_two<GPTQ_F16>(x, y);
        }
        *(u32v4*)(to + (int64_t)i * a.ldt) = o;
    }
}

// Tiles behind the last full round are cut along K so that their pieces fill rounds: what that takes is counted in
// steps of K (1.7 us), a piece's own at 8 beside its steps, its 256 KB of sums written and joined at 0.065.
// Measured: 160 tiles of 544 steps uncut 802 us, in three pieces 600.
inline DensePlan dense16_plan(int64_t t, int64_t rows, int64_t ldx) {
    DensePlan p;
    p.tiles_r = (rows + kTileR - 1) / kTileR;
    p.tiles_t = (t + kTileT - 1) / kTileT;
    p.tiles = p.tiles_r * p.tiles_t;
    const int64_t rest = p.tiles % kCUs, steps = ldx / kTileK;
    p.splits = 1;
    double best = (double)(steps + 8);
    for (int64_t s = 2; rest && s <= steps / kSplitSteps && s <= 32; ++s) {
        const double cost = (double)((rest * s + kCUs - 1) / kCUs) * ((double)((steps + s - 1) / s) + 8.0) + 0.065 * (double)(rest * s);
        if (cost < 0.97 * best) {
            best = cost;
            p.splits = s;
        }
    }
    p.whole = p.splits > 1 ? p.tiles - rest : p.tiles;
    return p;
}

constexpr int64_t kTokens16 = 1 << 14;  // tokens that the workspace holds operands of at once

}  // namespace gptq
