// linear_dense.hpp -- the product with codes for many tokens: weights decoded once to 16 bits, then a
// tiled MFMA product with the epilogue of linear.hip in it.
//
// decode_kernel writes W^ [rows, ldw] in the call's 16-bit type, ldw = n rounded up to 64, zeros
// behind n.  In f16 the power of two of a row's largest scale is taken out (row_power) and put
// back on the f32 sums, so that no scale overflows and only weights 2^-14 of the row's largest lose
// bits.  One read of the codes, one write of 2 bytes a weight: 39 us for 5120 x 17408, 6.0 TB/s.  That
// rounding to 16 bits (half a step a weight, as the activations have) buys the matrix units' whole rate;
// the exact sums of linear_tile_kernel stop at half of it, one f32 multiply-add for every 32 products.
//
// dense_kernel: 256 tokens x 256 rows a workgroup, 8 waves of 128 tokens x 64 rows, K in steps of 64
// through two LDS buffers filled by 16-byte loads straight to LDS.  A lane's 16 bytes are k
// neighbours of one row, which is what a 16x16x32 operand wants, so LDS keeps rows of 128 bytes whose
// eight 16-byte pieces are permuted by the row's low bits (the loads permute them on the way in),
// and the operand reads touch all banks.  W is operand A: an output's four registers are then four
// neighbouring columns of Y, stored as one vector.  Bound by the matrix units: 4096 tokens of 5120 x 17408
// take 573 us, 1270 TFLOP/s (MFMA in 64 % of a SIMD's cycles by the hardware's counters), and 26 us to join the 64 tiles behind the last full round (the library's
// product of decoded operands 673 us, without decoding and epilogue).
#pragma once
#include "linear_codes.hpp"

namespace gptq {

constexpr int kTileT = 256, kTileR = 256, kTileK = 64;
constexpr int kDenseWaves = 8;

struct DenseArgs {
    LinArgs l;
    const uint16_t* W;     // decoded weights [rows, ldw]
    const float* power;    // f16: 2^e of each row, taken out of W
    int ldw;               // n rounded up to kTileK
    int n;
    int tiles_r, tiles;    // tiles along the rows of W, tiles in all
    int whole, splits;     // tiles taken whole; the others are cut along K into `splits` pieces
    float* part;           // [tiles - whole][splits] pieces of 256 x 256 sums
};

// Rounds of 256 tiles (one a CU) run whole.  The tiles behind the last full round would leave CUs
// idle, so they are cut along K into as many pieces as there are CUs for, of at least kSplitSteps steps;
// the pieces' sums go through memory and dense_join_kernel adds them in order.  (Adding them in the
// workgroup that arrives last needs a release of its XCD's L2 by every piece: 8 x 32 of them took 80 us.)
constexpr int kSplitSteps = 6;
struct DensePlan {
    int64_t tiles_r, tiles_t, tiles, whole, splits;
};
inline DensePlan dense_plan(int64_t t, int64_t rows, int64_t n) {
    DensePlan p;
    p.tiles_r = (rows + kTileR - 1) / kTileR;
    p.tiles_t = (t + kTileT - 1) / kTileT;
    p.tiles = p.tiles_r * p.tiles_t;
    const int64_t rest = p.tiles % kCUs, steps = (n + kTileK - 1) / kTileK;
    p.splits = 1;
    if (rest) {
        p.splits = kCUs / rest < steps / kSplitSteps ? kCUs / rest : steps / kSplitSteps;
        if (p.splits < 2) p.splits = 1;
    }
    p.whole = p.splits > 1 ? p.tiles - rest : p.tiles;
    return p;
}

template <int DT>
__device__ __forceinline__ f32v4 mfma_dense(u32v4 a, u32v4 b, f32v4 c) {
    if constexpr (DT == GPTQ_F16) {
        typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    } else {
        return mfma16(a, b, c);
    }
}

// The power of two of the largest of n scales (a workgroup of 256, every lane's answer): top 2^-e in [1/2, 1);
// a row of zeros, or with an infinite scale, keeps e = 0.  |e| is held to 126 so that both powers are normal
// numbers.  part: four floats of LDS.
__device__ __forceinline__ int row_exponent(const float* sp, int n, float* part) {
    float top = 0.0f;
    for (int g = threadIdx.x; g < n; g += 256) top = fmaxf(top, fabsf(sp[g]));
#pragma unroll
    for (int k = 1; k < 64; k *= 2) top = fmaxf(top, __shfl_xor(top, k));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    int e = 0;
    if (top > 0.0f && top < INFINITY) e = min(max(ilogbf(top) + 1, -126), 126);
    return e;
}
// The level of the code in the low bits of w, and two values in the type, side by side.
template <int BITS>
__device__ __forceinline__ float level(uint32_t w) {
    return BITS == 4 ? (float)((int)(w & 15u) - 8) : (float)(w & 3u) - 1.5f;
}
template <int DT>
__device__ __forceinline__ uint32_t pack_two(float a, float b) {
    if constexpr (DT == GPTQ_BF16) {
        return round_bf16x2(a, b);
    } else {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        const h2 p = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, p);
    }
}
// x less its rounding to f16; 0 where that is not finite.
__device__ __forceinline__ float what_f16_leaves(float x) {
    const float r = x - (float)(_Float16)x;
    return r == r ? r : 0.0f;
}
// A row of W, G groups, times `less`, and zeros up to ldw: eight columns a thread.  TWO: as two terms, the second what
// the first's rounding leaves (nothing of values that are not finite), kTileK columns of each in turn.
template <int DT, int BITS, bool TWO = false>
__device__ __forceinline__ void decode_row(const uint8_t* cp, const float* sp, int G, float less, uint16_t* W, int ldw) {
    for (int u = threadIdx.x; u < ldw / 8; u += 256) {
        u32v4 out = {0u, 0u, 0u, 0u}, rest = {0u, 0u, 0u, 0u};
        if (u < G * 4) {
            const float s = sp[u >> 2] * less;
            uint32_t w = BITS == 4 ? ((const uint32_t*)cp)[u] : (uint32_t)((const uint16_t*)cp)[u];
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = level<BITS>(w) * s;
                w >>= BITS;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) out[k] = pack_two<DT>(v[2 * k], v[2 * k + 1]);
            if constexpr (TWO)
#pragma unroll
                for (int k = 0; k < 4; ++k) rest[k] = pack_two<DT>(what_f16_leaves(v[2 * k]), what_f16_leaves(v[2 * k + 1]));
        }
        if constexpr (TWO) {
            uint16_t* to = W + (8 * u / kTileK) * (2 * kTileK) + 8 * u % kTileK;
            *(u32v4*)to = out;
            *(u32v4*)(to + kTileK) = rest;
        } else {
            *(u32v4*)(W + 8 * u) = out;
        }
    }
}

// One workgroup per row of W.
template <int DT, int BITS>
__global__ __launch_bounds__(256) void decode_kernel(LinArgs a, uint16_t* W, float* power, int ldw) {
    const int64_t row = blockIdx.x;
    const float* sp = a.scale + row * a.G;
    float less = 1.0f;
    if constexpr (DT == GPTQ_F16) {
        __shared__ float part[4];
        const int e = row_exponent(sp, a.G, part);
        less = ldexpf(1.0f, -e);
        if (threadIdx.x == 0) power[row] = ldexpf(1.0f, e);
    }
    decode_row<DT, BITS>(a.codes + row * a.G * (4 * BITS), sp, a.G, less, W + row * ldw, ldw);
}

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;

// Sixteen bytes a lane from base (the same in the wave) + off bytes to 1 KB of LDS.
__device__ __forceinline__ void load_to_lds(const uint16_t* base, uint32_t off, uint16_t* lds) {
    __builtin_amdgcn_global_load_lds((global_void*)((const char*)base + off), (lds_void*)lds, 16, 0, 0);
}

// The operand registers of row r, 16-byte piece p of a tile in LDS.
__device__ __forceinline__ u32v4 tile_piece(const uint16_t* lds, int r, int p) {
    return *(const u32v4*)(lds + r * kTileK + ((p ^ (r & 7)) << 3));
}

struct Pieces {
    u32v4 w[4], x[8];
};
// A wave's operands of half kk of a step.
__device__ __forceinline__ void dense_read(const uint16_t* xs, const uint16_t* ws, int kk, int c, int h, int wt, int wr,
                                           Pieces& p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p.w[i] = tile_piece(ws, wr * 64 + i * 16 + c, kk * 4 + h);
#pragma unroll
    for (int j = 0; j < 8; ++j) p.x[j] = tile_piece(xs, wt * 128 + j * 16 + c, kk * 4 + h);
}
template <int DT>
__device__ __forceinline__ void dense_mul(const Pieces& p, f32v4 (&acc)[4][8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = mfma_dense<DT>(p.w[i], p.x[j], acc[i][j]);
}
// The reads of the next operands in between the products of the present ones.
__device__ __forceinline__ void dense_interleave() {
#pragma unroll
    for (int k = 0; k < 12; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 8, 0);
}

// A tile's sums over steps first .. steps - 1 of `all`: 256 rows of X from tok0 on (its last, t - 1, stands for
// those behind it) by 256 of W from row0 on, in this wave's registers.  n: the columns of X that are there.  XS, WS: a
// tile of X, of W, is that of 2^XS, 2^WS steps in a row, the terms of the other operand.
template <int DT, int XS = 0, int WS = 0>
__device__ __forceinline__ void dense_sums(const uint16_t* X, int64_t ldx, int t, int tok0, const uint16_t* W, int ldw,
                                           int row0, int n, int first, int steps, int all, uint16_t* xs0, uint16_t* ws0,
                                           uint16_t* xs1, uint16_t* ws1, f32v4 (&acc)[4][8]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int wt = wave >> 2, wr = wave & 3;
    // A wave's load i fills rows 32 wave + 8 i .. + 7 of a tile, lane l the piece l % 8 of row l / 8.
    // Offsets are bytes from the tile's first row, below 2^32 for rows of up to 2^22 elements; W has
    // rows up to a whole tile.
    const int sub = lane >> 3, piece = ((lane & 7) ^ sub) * 8;
    X += (int64_t)tok0 * ldx;
    W += (int64_t)(row0 + wave * 32) * ldw;
    uint32_t xo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        xo[i] = 2u * ((uint32_t)min(wave * 32 + i * 8 + sub, t - 1 - tok0) * (uint32_t)ldx + (uint32_t)piece);
    const uint32_t wo = 2u * ((uint32_t)sub * (uint32_t)ldw + (uint32_t)piece);
    // The last step may hold 32 columns: its other pieces of X are read from the token's own values (W
    // has zeros there).
    const uint32_t back = (n % kTileK) && piece >= 32 ? 64u : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = f32v4{0.f, 0.f, 0.f, 0.f};

    auto load = [&](int s, uint16_t* xs, uint16_t* ws) {
        const uint32_t less = s == all - 1 ? back : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            load_to_lds(X + (int64_t)(s >> XS) * kTileK, xo[i] - less, xs + (wave * 32 + i * 8) * kTileK);
            load_to_lds(W + (int64_t)(s >> WS) * kTileK + (int64_t)i * 8 * ldw, wo, ws + (wave * 32 + i * 8) * kTileK);
        }
        // Ahead of the step's products (the scheduler would sink the loads to the barrier).
        __builtin_amdgcn_sched_barrier(0);
    };
    // A step's second half is read while its first is multiplied, the next step's first half while the
    // second is; the one barrier a step stands between, when the step's tile is read out and the
    // next one is there.  Loads run two steps ahead.
    Pieces p0, p1;
    // Behind the last step the last tile is loaded and read again, to nothing, so that the loop has no
    // branches.
    auto step = [&](int s, uint16_t* xs, uint16_t* ws, uint16_t* xn, uint16_t* wn) {
        dense_read(xs, ws, 1, c, h, wt, wr, p1);
        dense_mul<DT>(p0, acc);
        dense_interleave();
        __syncthreads();
        load(min(s + 2, steps - 1), xs, ws);
        dense_read(xn, wn, 0, c, h, wt, wr, p0);
        dense_mul<DT>(p1, acc);
        dense_interleave();
    };
    load(first, xs0, ws0);
    __syncthreads();
    load(min(first + 1, steps - 1), xs1, ws1);
    dense_read(xs0, ws0, 0, c, h, wt, wr, p0);
    int s = first;
    for (; s + 1 < steps; s += 2) {
        step(s, xs0, ws0, xs1, ws1);
        step(s + 1, xs1, ws1, xs0, ws0);
    }
    if (s < steps) step(s, xs0, ws0, xs1, ws1);
    __syncthreads();
}

template <int DT>
__global__ __launch_bounds__(kDenseWaves * 64) void dense_kernel(DenseArgs a) {
    __shared__ __attribute__((aligned(16))) uint16_t xs0[kTileT * kTileK];
    __shared__ __attribute__((aligned(16))) uint16_t ws0[kTileR * kTileK];
    __shared__ __attribute__((aligned(16))) uint16_t xs1[kTileT * kTileK];
    __shared__ __attribute__((aligned(16))) uint16_t ws1[kTileR * kTileK];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int wt = wave >> 2, wr = wave & 3;
    int tile = blockIdx.x, split = 0;
    const bool cut = tile >= a.whole;
    if (cut) {
        split = (tile - a.whole) % a.splits;
        tile = a.whole + (tile - a.whole) / a.splits;
    }
    const int tok0 = tile / a.tiles_r * kTileT, row0 = tile % a.tiles_r * kTileR;
    const int all = a.ldw / kTileK;
    const int first = cut ? (int)((int64_t)all * split / a.splits) : 0;
    const int steps = cut ? (int)((int64_t)all * (split + 1) / a.splits) : all;
    f32v4 acc[4][8];
    dense_sums<DT>((const uint16_t*)a.l.X, a.l.ldx, a.l.t, tok0, a.W, a.ldw, row0, a.n, first, steps, all, xs0, ws0, xs1, ws1, acc);

    // Epilogue by way of LDS, 64 x 64 outputs of a wave at a time: a lane then has 16 neighbouring
    // columns of one token, four lanes 128 bytes of Y, and the activation's code is there once.
    if (cut) {  // a piece's sums to memory, a lane's registers side by side with its neighbours'
        float* mine = a.part + ((int64_t)(tile - a.whole) * a.splits + split) * (kTileT * kTileR);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *(f32v4*)(mine + ((i * 8 + j) * (kDenseWaves * 64) + threadIdx.x) * 4) = acc[i][j];
        return;
    }
    float* buf = (float*)(wave < 2 ? xs0 : wave < 4 ? ws0 : wave < 6 ? xs1 : ws1) + (wave & 1) * 4096;
    const int r0 = row0 + wr * 64 + (lane & 3) * 16;
    // Rows of Y (and of the residual) that keep 16-byte vectors aligned; at others 16 columns a lane, stored one
    // by one, cost more (2500 tokens of 2500 x 512: 47 us against 32).
    const bool aligned = a.l.ldy % 8 == 0 && ((uintptr_t)a.l.Y & 15u) == 0 &&
                         (!a.l.R || (a.l.ldr % 8 == 0 && ((uintptr_t)a.l.R & 15u) == 0));
    const bool vec = r0 + 16 <= a.l.rows;
    float b[16], p[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int r = min(aligned ? r0 + v : row0 + wr * 64 + lane, a.l.rows - 1);
        b[v] = a.l.bias ? a.l.bias[r] : 0.0f;
        p[v] = DT == GPTQ_F16 ? a.power[r] : 1.0f;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(f32v4*)(buf + (j * 16 + c) * 64 + (((i * 4 + h) ^ c) << 2)) = acc[i][half * 4 + j];
        __builtin_amdgcn_wave_barrier();
        if (!aligned) {  // a column a lane, four tokens at a time: neighbours store side by side
            const int r = row0 + wr * 64 + lane;
#pragma unroll 1
            for (int q = 0; q < 16; ++q) {
                const int tok = tok0 + wt * 128 + half * 64 + q * 4;
                float z[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int tt = q * 4 + v;
                    const float y = buf[tt * 64 + (((lane >> 2) ^ (tt & 15)) << 2) + (lane & 3)];
                    z[v] = DT == GPTQ_F16 ? fmaf(y, p[0], b[0]) : y + b[0];
                }
                activate_all(z, a.l.act);
                if (r >= a.l.rows) continue;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    if (tok + v >= a.l.t) break;
                    if (a.l.R) z[v] += load_one<DT>(a.l.R, (int64_t)(tok + v) * a.l.ldr + r);
                    store_one<DT>(a.l.Y, (int64_t)(tok + v) * a.l.ldy + r, z[v]);
                }
            }
            __builtin_amdgcn_wave_barrier();
            continue;
        }
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            const int tt = q * 16 + (lane >> 2), tok = tok0 + wt * 128 + half * 64 + tt;
            float z[16];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const f32v4 y = *(const f32v4*)(buf + tt * 64 + ((((lane & 3) * 4 + u) ^ (tt & 15)) << 2));
#pragma unroll
                for (int v = 0; v < 4; ++v) z[4 * u + v] = y[v];
            }
            if (tok >= a.l.t) continue;
#pragma unroll
            for (int v = 0; v < 16; ++v) z[v] = DT == GPTQ_F16 ? fmaf(z[v], p[v], b[v]) : z[v] + b[v];
            activate_all(z, a.l.act);
            const int64_t yo = (int64_t)tok * a.l.ldy + r0, ro = (int64_t)tok * a.l.ldr + r0;
            if (vec) {
                if (a.l.R) {
                    float r[8];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        load_eight<DT>(a.l.R, ro + 8 * u, r);
#pragma unroll
                        for (int v = 0; v < 8; ++v) z[8 * u + v] += r[v];
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) store_eight<DT>(a.l.Y, yo + 8 * u, z + 8 * u);
            } else {
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    if (r0 + v < a.l.rows)
                        store_one<DT>(a.l.Y, yo + v, a.l.R ? z[v] + load_one<DT>(a.l.R, ro + v) : z[v]);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// The sums of a cut tile's pieces, in their order, and the epilogue: four columns of a token a thread, in
// the order the pieces were written.
template <int DT>
__global__ __launch_bounds__(256) void dense_join_kernel(DenseArgs a) {
    constexpr int T = kDenseWaves * 64;
    const int tile = a.whole + blockIdx.y;
    const int u = blockIdx.x * 256 + threadIdx.x, thread = u % T, i = u / T >> 3, j = u / T & 7;
    const int lane = thread & 63, wave = thread >> 6;
    const int row = tile % a.tiles_r * kTileR + (wave & 3) * 64 + i * 16 + 4 * (lane >> 4);
    const int tok = tile / a.tiles_r * kTileT + (wave >> 2) * 128 + j * 16 + (lane & 15);
    if (tok >= a.l.t || row >= a.l.rows) return;
    const float* p = a.part + (int64_t)blockIdx.y * a.splits * (kTileT * kTileR) + 4 * u;
    f32v4 z = *(const f32v4*)p;
    for (int s = 1; s < a.splits; ++s) z += *(const f32v4*)(p + (int64_t)s * (kTileT * kTileR));
#pragma unroll
    for (int v = 0; v < 4; ++v)
        if (row + v < a.l.rows) finish<DT>(a.l, tok, row + v, DT == GPTQ_F16 ? z[v] * a.power[row + v] : z[v]);
}

}  // namespace gptq
