// linear.hip -- Y = act(X W^T + bias) + residual from the sweeps' codes on gfx950.
//
// W[r][j] = (q[r][j] - z) s[r][j / 32], z = 8 for q4tp's nibbles and 1.5 for q2tp's 2-bit codes,
// so a group of 32 columns adds s (sum_j q_j x_j - z sum_j x_j) to an output.  One 16x16x32 MFMA is
// one group: A = 16 tokens of X, B = the codes of 16 rows as whole numbers (codes16.hpp), and
// the result, exact up to f32 sums, is scaled by the lane's own s (D's column is the row of W)
// into the accumulator.  z and the operand's offset come out through the start value of D: X times
// a constant operand.  f16 and f32 X enter as two and three exact bf16 terms.
//
// Three layouts, chosen by codes_plan and linear_dense further down, which hold both sides' times:
//   linear_codes_kernel  few tokens, or few rows: bound by the read of the codes;
//   linear_tile_kernel   up to 256 tokens, smaller products and f32 at any number: bound by unpacking and scaling;
//   linear_dense.hpp     the rest: bound by the matrix units.
#include "../../include/gptq_check.h"
#include "check.hpp"
#include "codes16.hpp"
#include "common.hpp"

namespace gptq {

struct LinArgs {
    const void* X;
    int64_t ldx;
    const uint8_t* codes;
    const float* scale;
    const float* bias;
    const void* R;
    int64_t ldr;
    void* Y;
    int64_t ldy;
    int t, rows, G;  // G = n / 32 groups
    int act;
    float* part;     // [splits, t, rows] sums of pieces of K, or NULL: one piece, finished in place
};

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == GPTQ_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if constexpr (ACT == GPTQ_ACT_SILU) return z / (1.0f + expf(-z));
    // Forms that keep their relative precision for negative z: 1 + erf and 1 + tanh cancel there (5 % off at
    // z = -5, nothing left at -6).  erfc costs 8 us at 4096 tokens of 5120 x 2048 in bf16 (125 against 117), at
    // fewer nothing that shows.
    if constexpr (ACT == GPTQ_ACT_GELU) return 0.5f * z * erfcf(z * -0.70710678118654752f);
    if constexpr (ACT == GPTQ_ACT_GELU_TANH)
        return z / (1.0f + expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
    return z;
}
// The activation of N values, its kind looked at once.
template <int N>
__device__ __forceinline__ void activate_all(float (&z)[N], int act) {
    switch (act) {
        case GPTQ_ACT_RELU:
#pragma unroll
            for (int v = 0; v < N; ++v) z[v] = activate<GPTQ_ACT_RELU>(z[v]);
            break;
        case GPTQ_ACT_SILU:
#pragma unroll
            for (int v = 0; v < N; ++v) z[v] = activate<GPTQ_ACT_SILU>(z[v]);
            break;
        case GPTQ_ACT_GELU:
#pragma unroll
            for (int v = 0; v < N; ++v) z[v] = activate<GPTQ_ACT_GELU>(z[v]);
            break;
        case GPTQ_ACT_GELU_TANH:
#pragma unroll
            for (int v = 0; v < N; ++v) z[v] = activate<GPTQ_ACT_GELU_TANH>(z[v]);
            break;
        default: break;
    }
}

// Bias, activation, residual and the one rounding of an output.
template <int DT>
__device__ __forceinline__ void finish(const LinArgs& a, int tok, int r, float z) {
    float y[1] = {a.bias ? z + a.bias[r] : z};
    activate_all(y, a.act);
    if (a.R) y[0] += load_one<DT>(a.R, (int64_t)tok * a.ldr + r);
    store_one<DT>(a.Y, (int64_t)tok * a.ldy + r, y[0]);
}

// Word j of each lane of a wave's quarter h <- word h of quarter j.
__device__ __forceinline__ void transpose_quarters(uint32_t (&w)[4]) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w[0] = c[0];
    w[1] = c[1];
    w[2] = d[0];
    w[3] = d[1];
}

template <int BITS>
struct Code;
template <>
struct Code<4> {
    static constexpr int kBytes = 16;  // a group's
    static constexpr uint32_t kOffset = kMinus24;
    static constexpr float kShift = 24.0f;
    __device__ static void load(const uint8_t* p, uint32_t (&w)[4]) {
        const u32v4 v = *(const u32v4*)p;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = v[j];
    }
    // Columns (k, k + 4) of a word's eight.
    __device__ static u32v4 operand(uint32_t w) { return unpack_nibbles(w); }
};
template <>
struct Code<2> {
    static constexpr int kBytes = 8;
    static constexpr uint32_t kOffset = 0xC0B0C0B0u;  // bf16's -5.5 = -(4 + 1.5)
    static constexpr float kShift = 5.5f;
    __device__ static void load(const uint8_t* p, uint32_t (&w)[4]) {
        const u32v2 v = *(const u32v2*)p;
        w[0] = v[0];
        w[1] = v[0] >> 16;
        w[2] = v[1];
        w[3] = v[1] >> 16;
    }
    // Low 16 bits: columns 0..3 to the low half, 4..7 to the high one; 4 + q has q in bits 5, 6.
    __device__ static u32v4 operand(uint32_t w) {
        const uint32_t x = __builtin_amdgcn_perm(0u, w, 0x0c010c00u);
        return u32v4{and_or(x << 5, 0x00600060u, 0x40804080u), and_or(x << 3, 0x00600060u, 0x40804080u),
                     and_or(x << 1, 0x00600060u, 0x40804080u), and_or(x >> 1, 0x00600060u, 0x40804080u)};
    }
};

// The scales of a quad, one group in each quarter of the wave: s[j] <- quarter j's, in every lane.
__device__ __forceinline__ void spread_quarters(float x, float (&s)[4]) {
    const uint32_t u = __float_as_uint(x);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
    s[0] = __uint_as_float(b[0]);
    s[1] = __uint_as_float(b[1]);
    s[2] = __uint_as_float(c[0]);
    s[3] = __uint_as_float(c[1]);
}

// Four groups of the rows of a lane as they are loaded, one group a quarter of the wave: codes, not yet
// transposed, and scales, not yet spread (a quarter loads the scale of its own group only).
// A group that is not there (the last quad may hold fewer than four) has scale 0.
template <int BITS, int RT>
struct Quad {
    uint32_t w[RT][4];
    float s[RT];
    __device__ void load(const uint8_t* const (&cp)[RT], const float* const (&sp)[RT], int q, int h, int G) {
        const int g = 4 * q + h, gc = min(g, G - 1);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            Code<BITS>::load(cp[i] + (int64_t)gc * Code<BITS>::kBytes, w[i]);
            s[i] = sp[i][gc];
            if (g >= G) s[i] = 0.0f;
        }
    }
};

// A workgroup owns 16 RT rows of W and 16 TT tokens; its NW waves take quads of four groups in turn and
// their sums are joined in LDS, where the epilogue runs.  Per quad a lane loads 16 bytes (q4tp), one group
// of its row; a 4 x 4 transpose over the quarters of the wave (four permlane swaps) hands each quarter its
// eight columns of every group.  Bound by latency rather than bytes or instructions: 13 tokens of
// 5120 x 17408 take 27.3 us with the join, 2.1 TB/s of codes and scales (a copy reaches 4.9); by the
// hardware's counters vector instructions are in 39 % of a SIMD's cycles and MFMA in 11 %, and a wave, which
// makes 23 loads in all, waits for them or its turn for four fifths of its time.
//
// PD: quads in flight a wave.  Loads return in order, so a quad's codes, scales and activations are
// loaded together, all PD quads ahead of their use.
template <int DT, int BITS, int RT, int TT, int NW, int PD>
__global__ __launch_bounds__(NW * 64) void linear_codes_kernel(LinArgs a) {
    constexpr int NT = kTerms<DT>;
    __shared__ float red[NW][RT * TT * 4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int row0 = blockIdx.x * 16 * RT, tok0 = blockIdx.y * 16 * TT;
    const uint8_t* cp[RT];
    const float* sp[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int64_t row = min(row0 + 16 * i + c, a.rows - 1);
        cp[i] = a.codes + row * a.G * Code<BITS>::kBytes;
        sp[i] = a.scale + row * a.G;
    }
    int64_t xo[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) xo[tt] = (int64_t)min(tok0 + tt * 16 + c, a.t - 1) * a.ldx + 8 * h;
    f32v4 acc[RT][TT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) acc[i][tt] = f32v4{0.f, 0.f, 0.f, 0.f};
    const u32v4 offset = {Code<BITS>::kOffset, Code<BITS>::kOffset, Code<BITS>::kOffset, Code<BITS>::kOffset};

    // This workgroup's quads: all, or piece blockIdx.z of K.
    const int all = (a.G + 3) >> 2;
    const int first = (int)((int64_t)all * blockIdx.z / gridDim.z) + wave;
    const int quads = (int)((int64_t)all * (blockIdx.z + 1) / gridDim.z);
    Quad<BITS, RT> w[PD];
    Raw<DT> x[PD][4][TT];
    auto load = [&](int p, int q) {
        w[p].load(cp, sp, q, h, a.G);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) x[p][j][tt].load(a.X, xo[tt] + 32 * min(4 * q + j, a.G - 1));
    };
#pragma unroll
    for (int p = 0; p < PD; ++p)
        if (first + p * NW < quads) load(p, first + p * NW);
    for (int q0 = first; q0 < quads; q0 += PD * NW) {
#pragma unroll
        for (int p = 0; p < PD; ++p) {
            const int q = q0 + p * NW;
            if (q >= quads) break;
            float s[RT][4];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                transpose_quarters(w[p].w[i]);
                spread_quarters(w[p].s[i], s[i]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (4 * q + j >= a.G) break;  // the same in every lane
                u32v4 code[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i) code[i] = Code<BITS>::operand(w[p].w[i][j]);
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) {
                    u32v4 t[NT];
                    raw_terms<DT>(x[p][j][tt].a, t);
                    f32v4 start = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < NT; ++k) start = mfma16(t[k], offset, start);
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        f32v4 d = start;
#pragma unroll
                        for (int k = 0; k < NT; ++k) d = mfma16(t[k], code[i], d);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][tt][r] = fmaf(s[i][j], d[r], acc[i][tt][r]);
                    }
                }
            }
            if (q + PD * NW < quads) load(p, q + PD * NW);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wave][(i * TT + tt) * 4 + r][lane] = acc[i][tt][r];
    __syncthreads();
    for (int u = wave; u < RT * TT * 4; u += NW) {
        float z = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) z += red[k][u][lane];
        const int tok = tok0 + (u >> 2) % TT * 16 + 4 * h + (u & 3), r = row0 + (u >> 2) / TT * 16 + c;
        if (tok < a.t && r < a.rows) {
            if (a.part)
                a.part[((int64_t)blockIdx.z * a.t + tok) * a.rows + r] = z;
            else
                finish<DT>(a, tok, r, z);
        }
    }
}

// linear_tile_kernel: the same sums with the waves side by side on rows.  A workgroup owns 128 RT rows
// of W (16 RT a wave), 16 TT tokens and a piece of K; the activations of KC quads at a time are split
// into their terms once, in operand order, into LDS (f16, f32: next to each group's start value), and every wave
// reads them from there while the next ones are on their way.  A wave's codes and scales run up to two
// quads ahead.  In bf16 the start value is an MFMA of its own, the same for the wave's RT row tiles: 128
// tokens of 5120 x 17408 take 66.7 us, 344 TFLOP/s, 70.9 with sums kept in LDS.  That is half vector
// instructions around the products (four multiply-adds and the unpacking per MFMA: 40 % of a SIMD's cycles by the
// hardware's counters, MFMA 23 %) and half waits, for the chunk's barrier, loads and LDS.
constexpr int kTileWaves = 8;

template <int DT, int BITS, int RT, int TT>
__global__ __launch_bounds__(kTileWaves * 64) void linear_tile_kernel(LinArgs a) {
    constexpr int NT = kTerms<DT>;
    constexpr int KC = (NT == 3 ? 4 : 8) / TT;       // quads of a chunk
    constexpr int F = KC * 4 * TT;                   // 16-token operands of a chunk (one group each)
    constexpr int FT = F / kTileWaves;               // .. that a wave prepares
    constexpr int PD = KC < 2 ? 1 : 2;               // quads of codes in flight; KC is a multiple of it
    __shared__ u32v4 xs[2][F][NT][64];
    __shared__ f32v4 start[2][NT > 1 ? F : 1][4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int row0 = (blockIdx.x * kTileWaves + wave) * 16 * RT, tok0 = blockIdx.y * 16 * TT;
    const int all = (a.G + 3) >> 2;
    const int first = (int)((int64_t)all * blockIdx.z / gridDim.z), end = (int)((int64_t)all * (blockIdx.z + 1) / gridDim.z);
    const uint8_t* cp[RT];
    const float* sp[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int64_t row = min(row0 + 16 * i + c, a.rows - 1);
        cp[i] = a.codes + row * a.G * Code<BITS>::kBytes;
        sp[i] = a.scale + row * a.G;
    }
    // Operand f of a chunk: group f / TT of it, tokens 16 (f % TT) ..
    Raw<DT> raw[FT];
    auto fetch = [&](int q0) {
#pragma unroll
        for (int k = 0; k < FT; ++k) {
            const int f = wave * FT + k, g = min(4 * q0 + f / TT, a.G - 1);
            raw[k].load(a.X, (int64_t)min(tok0 + f % TT * 16 + c, a.t - 1) * a.ldx + 32 * g + 8 * h);
        }
    };
    auto prepare = [&](int buf) {
#pragma unroll
        for (int k = 0; k < FT; ++k) {
            const int f = wave * FT + k;
            u32v4 t[NT];
            float sum;
            raw_terms_sum<DT>(raw[k].a, t, sum);
#pragma unroll
            for (int n = 0; n < NT; ++n) xs[buf][f][n][lane] = t[n];
            if constexpr (NT > 1) {
                sum = quad_sum(sum);
                if (h == 0) ((float*)start[buf][f])[c] = sum * -Code<BITS>::kShift;
            }
        }
    };
    Quad<BITS, RT> w[PD];
    auto load = [&](int p, int q) { w[p].load(cp, sp, q, h, a.G); };
    f32v4 acc[RT][TT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) acc[i][tt] = f32v4{0.f, 0.f, 0.f, 0.f};
    if (first < end) {
        fetch(first);
#pragma unroll
        for (int p = 0; p < PD; ++p) load(p, min(first + p, end - 1));
        prepare(0);
    }
    __syncthreads();
    const u32v4 offset = {Code<BITS>::kOffset, Code<BITS>::kOffset, Code<BITS>::kOffset, Code<BITS>::kOffset};
    int buf = 0;
    for (int q0 = first; q0 < end; q0 += KC) {
        fetch(min(q0 + KC, end - 1));
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const int q = q0 + k;
            if (q >= end) break;
            uint32_t now[RT][4];
            float s[RT][4];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) now[i][j] = w[k % PD].w[i][j];
                spread_quarters(w[k % PD].s[i], s[i]);
                transpose_quarters(now[i]);
            }
            load(k % PD, min(q + PD, end - 1));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32v4 code[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i) code[i] = Code<BITS>::operand(now[i][j]);
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) {
                    const int f = (k * 4 + j) * TT + tt;
                    u32v4 x[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) x[n] = xs[buf][f][n][lane];
                    f32v4 d0 = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (NT == 1)
                        d0 = mfma16(x[0], offset, d0);
                    else
                        d0 = start[buf][f][h];
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        f32v4 d = d0;
#pragma unroll
                        for (int n = 0; n < NT; ++n) d = mfma16(x[n], code[i], d);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][tt][r] = fmaf(s[i][j], d[r], acc[i][tt][r]);
                    }
                }
            }
        }
        prepare(buf ^ 1);
        buf ^= 1;
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tok = tok0 + tt * 16 + 4 * h + r, row = row0 + 16 * i + c;
                if (tok >= a.t || row >= a.rows) continue;
                if (a.part)
                    a.part[((int64_t)blockIdx.z * a.t + tok) * a.rows + row] = acc[i][tt][r];
                else
                    finish<DT>(a, tok, row, acc[i][tt][r]);
            }
}

// The sums of the pieces of K, in their order, and the epilogue.
template <int DT>
__global__ __launch_bounds__(256) void linear_join_kernel(LinArgs a, int splits) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)a.t * a.rows;
    if (i >= n) return;
    float z = 0.0f;
    for (int s = 0; s < splits; ++s) z += a.part[s * n + i];
    const int tok = (int)(i / a.rows);
    finish<DT>(a, tok, (int)(i - (int64_t)tok * a.rows), z);
}

}  // namespace gptq

#include "linear_dense.hpp"

namespace gptq {

typedef void (*LinKernel)(LinArgs);
// How a product with few tokens, or in f32, is laid out: 16 rt rows and 16 tt tokens a wave; `waves` of a
// workgroup share them and cut K between them (linear_codes_kernel), or 0: kTileWaves side by side
// (linear_tile_kernel); K in `splits` pieces, joined by linear_join_kernel.
struct CodesPlan {
    int rt, tt, waves, splits;
};
// Measured (us, bf16 unless said otherwise; 4096 x 4096 / 5120 x 17408):
//   up to 16 tokens  one launch, 16 waves cutting K: 8.2 / 45.9; 8 waves of 32 rows and pieces of K for four
//                    workgroups a CU: 10.4 / 27.5.  The second pays behind 2^25 weights, where the
//                    matrix takes longer to read than the second launch costs.
//   one round        8 waves of 32 rows x 16 tokens, K uncut, where that is at most a workgroup a CU and 2^25
//                    weights.  Against side by side: 32 tokens 10.9 / 14.8, 40 of 2560 x 2560 7.8 / 17.3,
//                    128 of 1024 x 4096 in f32 15.2 / 24.6; at two a CU 18.4 / 19.4 (64 tokens), at four
//                    31.9 / 21.9, and 47 / 33.9 for 32 tokens of 5120 x 17408.
//   above            side by side, 32 or 64 tokens: 64 tokens 19.4 / 42.4, 128 tokens 21.9 / 66.7.
// Side by side, pieces of K fill the rounds of one workgroup a CU: at two a CU (24 pieces of 5120 x 17408) the
// pieces' sums cost more than the idle lanes (40.6 against 33.9 us).  1000 tokens of 2500 x 8192 in f32, 160
// workgroups, take 234 uncut and 176 in three pieces; of 5120 x 2048, 320 workgroups, 128 and 118.
static bool one_round(int64_t t, int64_t rows, int64_t n) {
    return rows * n <= ((int64_t)1 << 25) && (rows + 31) / 32 * ((t + 15) / 16) <= kCUs;
}
static CodesPlan codes_plan(int64_t t, int64_t rows, int64_t n) {
    const bool large = rows * n > ((int64_t)1 << 25);
    const int64_t quads = (n / 32 + 3) / 4, wide = (rows + 31) / 32;
    CodesPlan p;
    if (t <= 16 && !large)
        p = CodesPlan{1, 1, 16, 1};
    else if (t <= 16)
        p = CodesPlan{2, 1, 8, (int)((1024 + wide / 2) / wide)};
    else if (one_round(t, rows, n))
        p = CodesPlan{2, 1, 8, 1};
    else
        p = CodesPlan{2, t <= 32 ? 2 : 4, 0, 1};
    if (p.waves == 0) {
        const int64_t wg = (rows + 32 * kTileWaves - 1) / (32 * kTileWaves) * ((t + 16 * p.tt - 1) / (16 * p.tt));
        // Rounds of workgroups, a CU each, times the quads of a piece and what a piece costs beside them.
        double best = (double)((wg + kCUs - 1) / kCUs) * (double)quads;
        for (int64_t k = 2; k <= 64 && (k - 1) * wg < 3 * kCUs; ++k) {
            const double cost = (double)((k * wg + kCUs - 1) / kCUs) * ((double)((quads + k - 1) / k) + 2.0);
            if (cost < 0.95 * best) {
                best = cost;
                p.splits = (int)k;
            }
        }
    }
    if (p.splits > quads) p.splits = (int)quads;  // no empty piece
    if (p.splits < 1) p.splits = 1;
    return p;
}

template <int DT, int BITS>
static LinKernel codes_kernel(const CodesPlan& c) {
    if (c.waves == 16) return linear_codes_kernel<DT, BITS, 1, 1, 16, 2>;
    if (c.waves == 8) return linear_codes_kernel<DT, BITS, 2, 1, 8, 2>;
    return c.tt == 2 ? linear_tile_kernel<DT, BITS, 2, 2> : linear_tile_kernel<DT, BITS, 2, 4>;
}

}  // namespace gptq

using namespace gptq;

static bool linear_sizes_ok(int dtype, int64_t t, int64_t rows, int64_t n) {
    return dtype_size(dtype) && t >= 0 && t <= (1 << 24) && rows >= 1 && rows <= (1 << 23) &&
           t * rows <= ((int64_t)1 << 38) && n >= 32 && n <= (1 << 20) && n % 32 == 0;
}

// Many tokens in a 16-bit type run on decoded weights, where there is enough to multiply for three launches.
// Measured against linear_tile_kernel (us, dense / tile; rows x n):
//   bf16  200 tokens of 5120 x 17408 113 / 107, 400 of 5120 x 8192 77 / 122; 1000 of 1001 x 8192 (8e9 products)
//         43.0 / 45.0, of 2500 x 2048 (5e9) 37.6 / 38.4, of 1001 x 2048 (2e9) 26.4 / 23.4, of 2500 x 512 31 / 17.
//   f16   whose activations are two terms there: 1000 of 1001 x 2048 27.3 / 26.9, 400 of 1001 x 8192 (3e9)
//         35.1 / 35.5, 2500 of 2500 x 512 (3e9) 33 / 38, 400 of 5120 x 2048 44 / 48.
// Few rows stay with one_round: 512 tokens of 256 x 1024 18.4 / 4.1, of 256 x 16384 36.3 / 31.3.
// It rounds the weights, half a step each; GPTQ_EXACT_WEIGHTS keeps a call on linear_tile_kernel (bf16, 4096
// tokens of 5120 x 17408 1313 against 679, 1000 of 5120 x 8192 209 against 112).
static bool linear_dense(int dtype, int64_t t, int64_t rows, int64_t n) {
    const int64_t enough = dtype == GPTQ_BF16 ? 5000000000 : 2500000000;
    return dtype != GPTQ_F32 && t > 256 && t * rows * n > enough && !one_round(t, rows, n);
}
static int64_t dense_ld(int64_t n) { return round_up(n, kTileK); }
// Workspace of the dense product: the rows' powers of two, the weights (whole tiles of rows), the
// pieces' sums.
struct DenseSpace {
    size_t weights, part, bytes;
};
static DenseSpace dense_space(int64_t t, int64_t rows, int64_t n) {
    const DensePlan p = dense_plan(t, rows, n);
    DenseSpace s;
    s.weights = align256(sizeof(float) * (size_t)rows);
    s.part = s.weights + align256(2 * (size_t)round_up(rows, kTileR) * (size_t)dense_ld(n));
    s.bytes = s.part + sizeof(float) * (size_t)((p.tiles - p.whole) * p.splits) * (kTileT * kTileR);
    return s;
}

// A caller's dtype: the type, and whether its weights have to enter unrounded.
struct LinType {
    int dtype;
    bool exact;
};
static LinType linear_type(int dtype) { return LinType{dtype & ~GPTQ_EXACT_WEIGHTS, (dtype & GPTQ_EXACT_WEIGHTS) != 0}; }

extern "C" size_t gptq_linear_workspace_size(int type, int64_t t, int64_t rows, int64_t n) {
    const auto [dtype, exact] = linear_type(type);
    if (!linear_sizes_ok(dtype, t, rows, n) || t == 0) return 0;
    if (!exact && linear_dense(dtype, t, rows, n)) return dense_space(t, rows, n).bytes;
    const CodesPlan c = codes_plan(t, rows, n);
    return c.splits > 1 ? align256(sizeof(float) * (size_t)c.splits * (size_t)t * (size_t)rows) : 0;
}

template <int DT>
static int linear_dense_run(const LinArgs& l, bool four, int64_t n, void* workspace, hipStream_t st) {
    const DenseSpace sp = dense_space(l.t, l.rows, n);
    const DensePlan p = dense_plan(l.t, l.rows, n);
    char* ws = (char*)workspace;
    const DenseArgs d{l, (uint16_t*)(ws + sp.weights), (float*)ws, (int)dense_ld(n), (int)n,
                      (int)p.tiles_r, (int)p.tiles, (int)p.whole, (int)p.splits, (float*)(ws + sp.part)};
    const int64_t ldw = d.ldw, cb = four ? n / 2 : n / 4, cut = (p.tiles - p.whole) * p.splits;
    const int64_t sums = cut * kTileT * kTileR;
    uint16_t* W = (uint16_t*)d.W;
    float* power = (float*)d.power;
    {
        ProfScope ps(FAM_LINEAR, st, 0.0, (double)l.rows * (cb + 4 * l.G + 2 * ldw));
        GPTQ_LAUNCH(st, "linear_decode",
                    (four ? decode_kernel<DT, 4><<<(unsigned)l.rows, 256, 0, st>>>(l, W, power, d.ldw)
                          : decode_kernel<DT, 2><<<(unsigned)l.rows, 256, 0, st>>>(l, W, power, d.ldw)),
                    rd(l.codes, cb, l.rows, cb, 1), rd(l.scale, l.G, l.rows, l.G), wr(W, ldw, l.rows, ldw, 2),
                    wr(power, l.rows, DT == GPTQ_F16 ? 1 : 0, l.rows));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    ProfScope ps(FAM_LINEAR, st, 2.0 * (double)l.t * l.rows * n, 0.0);
    GPTQ_LAUNCH(st, "linear_dense",
                (dense_kernel<DT><<<(unsigned)(p.whole + cut), kDenseWaves * 64, 0, st>>>(d)),
                rd(l.X, l.ldx, l.t, n, 2), rd(W, ldw, round_up(l.rows, kTileR), ldw, 2),
                rd(power, l.rows, DT == GPTQ_F16 ? 1 : 0, l.rows),
                rd(l.bias ? l.bias : l.scale, l.rows, l.bias ? 1 : 0, l.rows),
                rd(l.R ? l.R : (const void*)l.scale, l.ldr, l.R ? l.t : 0, l.rows, 2), wr(l.Y, l.ldy, l.t, l.rows, 2),
                wr(d.part, sums, cut ? 1 : 0, sums));
    if (cut)
        GPTQ_LAUNCH(st, "linear_dense_join",
                    (dense_join_kernel<DT><<<dim3(kTileT * kTileR / 1024, (unsigned)(p.tiles - p.whole)), 256, 0, st>>>(d)),
                    rd(d.part, sums, 1, sums), rd(power, l.rows, DT == GPTQ_F16 ? 1 : 0, l.rows),
                    rd(l.bias ? l.bias : l.scale, l.rows, l.bias ? 1 : 0, l.rows),
                    rd(l.R ? l.R : (const void*)l.scale, l.ldr, l.R ? l.t : 0, l.rows, 2),
                    wr(l.Y, l.ldy, l.t, l.rows, 2));
    return GPTQ_OK;
}

extern "C" int gptq_linear(const void* X, int64_t ldx, int type, int64_t t, int codec,
                           const uint8_t* codes, const float* scale, int64_t rows, int64_t n,
                           const float* bias, int act, const void* residual, int64_t ldr, void* Y,
                           int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
    const auto [dtype, exact] = linear_type(type);
    if (!linear_sizes_ok(dtype, t, rows, n)) return GPTQ_EINVAL;
    if (codec != GPTQ_CODEC_Q4TP && codec != GPTQ_CODEC_Q2TP) return GPTQ_EINVAL;
    if (act < GPTQ_ACT_NONE || act > GPTQ_ACT_GELU_TANH) return GPTQ_EINVAL;
    if (t == 0) return GPTQ_OK;
    const int es = dtype_size(dtype);
    if (!X || !codes || !scale || !Y || ldx < n || ldx > (1 << 22) || ldx % (16 / es) != 0 || ldy < rows) return GPTQ_EINVAL;
    if (residual && ldr < rows) return GPTQ_EINVAL;
    if (!al16(X) || !al16(codes)) return GPTQ_EINVAL;
    // Elements at their natural alignment.
    if (((uintptr_t)Y | (uintptr_t)residual) % (unsigned)es || ((uintptr_t)scale | (uintptr_t)bias) % 4u)
        return GPTQ_EINVAL;
    const size_t need = gptq_linear_workspace_size(type, t, rows, n);
    if (need) {
        if (!workspace || workspace_bytes < need) return GPTQ_EWORKSPACE;
        if ((uintptr_t)workspace & 255u) return GPTQ_EINVAL;
    }
    const int64_t G = n / 32, cb = codec == GPTQ_CODEC_Q4TP ? n / 2 : n / 4;
    // Workgroups read their arguments at any time of the call: Y may be the residual (an output's own, read
    // before it is written) and nothing else.
    const RowSet y{Y, ldy * es, t, rows * es};
    auto whole = [](const void* p, int64_t bytes) { return RowSet{p, bytes, p ? 1 : 0, bytes}; };
    if (rows_meet(y, RowSet{X, ldx * es, t, n * es}) || rows_meet(y, whole(codes, rows * cb)) ||
        rows_meet(y, whole(scale, rows * G * 4)) || rows_meet(y, whole(bias, rows * 4)) ||
        rows_meet(y, whole(need ? workspace : nullptr, (int64_t)need)))
        return GPTQ_EINVAL;
    if (residual && !(residual == Y && (t == 1 || ldr == ldy)) && rows_meet(y, RowSet{residual, ldr * es, t, rows * es}))
        return GPTQ_EINVAL;
    CheckScope check;
    if (need) check_buffer(workspace, workspace_bytes, "workspace");
    check_buffer(X, (size_t)es * (size_t)((t - 1) * ldx + n), "X");
    check_buffer(codes, (size_t)(rows * cb), "codes");
    check_buffer(scale, sizeof(float) * (size_t)(rows * G), "scale");
    if (bias) check_buffer(bias, sizeof(float) * (size_t)rows, "bias");
    if (residual) check_buffer(residual, (size_t)es * (size_t)((t - 1) * ldr + rows), "residual");
    check_buffer(Y, (size_t)es * (size_t)((t - 1) * ldy + rows), "Y");
    hipStream_t st = (hipStream_t)stream;
    const LinArgs a{X, ldx, codes, scale, bias, residual, ldr, Y, ldy, (int)t, (int)rows, (int)G, act, nullptr};
    if (!exact && linear_dense(dtype, t, rows, n)) {
        const bool q4 = codec == GPTQ_CODEC_Q4TP;
        const int rc = dtype == GPTQ_BF16 ? linear_dense_run<GPTQ_BF16>(a, q4, n, workspace, st)
                                          : linear_dense_run<GPTQ_F16>(a, q4, n, workspace, st);
        if (rc != GPTQ_OK) return rc;
        if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
        return check.finish();
    }
    const CodesPlan ct = codes_plan(t, rows, n);
    const bool four = codec == GPTQ_CODEC_Q4TP;
    const LinKernel k =
        dtype == GPTQ_F32    ? (four ? codes_kernel<GPTQ_F32, 4>(ct) : codes_kernel<GPTQ_F32, 2>(ct))
        : dtype == GPTQ_BF16 ? (four ? codes_kernel<GPTQ_BF16, 4>(ct) : codes_kernel<GPTQ_BF16, 2>(ct))
                             : (four ? codes_kernel<GPTQ_F16, 4>(ct) : codes_kernel<GPTQ_F16, 2>(ct));
    void (*const join)(LinArgs, int) = dtype == GPTQ_F32    ? linear_join_kernel<GPTQ_F32>
                                       : dtype == GPTQ_BF16 ? linear_join_kernel<GPTQ_BF16>
                                                            : linear_join_kernel<GPTQ_F16>;
    // Grid y is limited to 65535; 2^24 tokens are launched in slices of 2^19.
    constexpr int64_t kSlice = 1 << 19;
    for (int64_t t0 = 0; t0 < t; t0 += kSlice) {
        LinArgs b = a;
        b.t = (int)(t - t0 < kSlice ? t - t0 : kSlice);
        b.X = (const char*)X + t0 * ldx * es;
        b.Y = (char*)Y + t0 * ldy * es;
        if (residual) b.R = (const char*)residual + t0 * ldr * es;
        if (ct.splits > 1) b.part = (float*)workspace;
        const int64_t tile_rows = 16 * ct.rt * (ct.waves ? 1 : kTileWaves);
        const dim3 grid((unsigned)((rows + tile_rows - 1) / tile_rows), (unsigned)((b.t + 16 * ct.tt - 1) / (16 * ct.tt)),
                        (unsigned)ct.splits);
        ProfScope ps(FAM_LINEAR, st, 2.0 * (double)b.t * rows * n, (double)rows * (cb + 4 * G));
        GPTQ_LAUNCH(st, "linear_codes", (k<<<grid, (ct.waves ? ct.waves : kTileWaves) * 64, 0, st>>>(b)), rd(b.X, ldx, b.t, n, es),
                    rd(codes, cb, rows, cb, 1), rd(scale, G, rows, G),
                    rd(bias ? (const void*)bias : (const void*)scale, rows, bias ? 1 : 0, rows),
                    rd(residual ? b.R : (const void*)scale, ldr, residual ? b.t : 0, rows, es),
                    wr(b.part ? (const void*)b.part : b.Y, b.part ? rows : ldy, b.part ? (int64_t)b.t * ct.splits : b.t, rows,
                       b.part ? 4 : es));
        if (b.part)
            GPTQ_LAUNCH(st, "linear_join",
                        (join<<<(unsigned)((b.t * rows + 255) / 256), 256, 0, st>>>(b, ct.splits)),
                        rd(b.part, rows, (int64_t)b.t * ct.splits, rows),
                        rd(bias ? (const void*)bias : (const void*)scale, rows, bias ? 1 : 0, rows),
                        rd(residual ? b.R : (const void*)scale, ldr, residual ? b.t : 0, rows, es),
                        wr(b.Y, ldy, b.t, rows, es));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}

extern "C" int gptq_check_linear_plan(int type, int64_t t, int64_t rows, int64_t n, int64_t* plan) {
    const auto [dtype, exact] = linear_type(type);
    if (!plan || !linear_sizes_ok(dtype, t, rows, n) || t == 0) return GPTQ_EINVAL;
    if (!exact && linear_dense(dtype, t, rows, n)) {
        const DensePlan p = dense_plan(t, rows, n);
        plan[0] = 3;
        plan[1] = p.splits;
        plan[2] = p.whole;
        plan[3] = p.tiles - p.whole;
        return GPTQ_OK;
    }
    const CodesPlan p = codes_plan(t, rows, n);
    plan[0] = p.waves ? 1 : 2;
    plan[1] = p.splits;
    plan[2] = plan[3] = 0;
    return GPTQ_OK;
}
