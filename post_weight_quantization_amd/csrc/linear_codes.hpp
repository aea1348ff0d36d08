// linear_codes.hpp -- kernels that multiply activations by the sweeps' codes as they are, and how a product is
// laid out on them: one matrix (linear.hip), or two side by side (gated.hip).
#pragma once
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
    float* part;     // [splits, t, sums] sums of pieces of K, or NULL: one piece, finished in place
    // EPI_GATED and EPI_GRAD: the second matrix, of the same sizes; EPI_GRAD: R is the gradient of Y.
    const uint8_t* codes2;
    const float* scale2;
    const float* bias2;
    int side;        // EPI_GRAD: columns of Y from the gate's gradients to the up projection's
};

// What becomes of the sums: Y = act(z + bias) + R; Y = act(a + bias) (b + bias2) of two matrices' sums; or, f32,
// the gradients of those a and b, side by side in Y, from that of act(a + bias) (b + bias2) in R.
enum { EPI_LINEAR = 0, EPI_GATED = 1, EPI_GRAD = 2 };
// Two matrices are multiplied as one whose rows are theirs in turns of 16: a tile of 16 rows and the next are
// the same rows of the first and the second, and a lane holds both sums of an output.
__host__ __device__ __forceinline__ constexpr int64_t sums_of(int epi, int64_t rows) {
    return epi == EPI_LINEAR ? rows : (rows + 15) / 16 * 32;
}
// Codes enter as their levels, without an offset, in f32 products of two matrices: beside the offset's part f32 sums
// lose two bits to four (a block of 2 tokens of 774 x 416 1.8e-6 off and 0.2e-6 without).  The unpacking takes three
// times the instructions, the products a third less.
template <int DT, int EPI>
constexpr bool kLevels = DT == GPTQ_F32 && EPI != EPI_LINEAR;
// Row of its matrix that row v of the sums is.
template <int EPI>
__device__ __forceinline__ int matrix_row(int v) {
    return EPI == EPI_LINEAR ? v : (v >> 5) * 16 + (v & 15);
}

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

// 1 / (1 + e^-z).  QUICK, for results of 16 bits: the hardware's power and reciprocal, off by 2^-23 and 2^-22, and an
// argument rounded once more, 2^-24 |z|; a quarter of the instructions.
template <bool QUICK>
__device__ __forceinline__ float logistic(float z) {
    if constexpr (QUICK) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
    return 1.0f / (1.0f + expf(-z));
}
// An activation and its slope.
template <int ACT, bool QUICK>
__device__ __forceinline__ float slope(float z, float& y) {
    if constexpr (ACT == GPTQ_ACT_SILU) {
        const float s = logistic<QUICK>(z);
        y = z * s;
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    if constexpr (ACT == GPTQ_ACT_GELU) {
        const float p = 0.5f * erfcf(z * -0.70710678118654752f);
        y = z * p;
        return fmaf(z * 0.39894228040143268f, expf(-0.5f * z * z), p);  // 1 / sqrt(2 pi)
    }
    if constexpr (ACT == GPTQ_ACT_GELU_TANH) {
        const float s = logistic<QUICK>(1.5957691216057308f * (z + 0.044715f * z * z * z));
        const float t = s * (1.0f - s);  // 0 far out, where z^2 may be infinite
        y = z * s;
        return t == 0.0f ? s : fmaf(z * t * 1.5957691216057308f, fmaf(0.134145f * z, z, 1.0f), s);
    }
    y = activate<ACT>(z);
    if constexpr (ACT == GPTQ_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    return 1.0f;
}
// a <- act(a) b, the activation's kind looked at once.
template <int ACT, bool QUICK, int N>
__device__ __forceinline__ void gate_of(float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int v = 0; v < N; ++v) {
        float y;
        slope<ACT, QUICK>(a[v], y);
        a[v] = y * b[v];
    }
}
template <bool QUICK, int N>
__device__ __forceinline__ void gate_all(float (&a)[N], const float (&b)[N], int act) {
    switch (act) {
        case GPTQ_ACT_RELU: gate_of<GPTQ_ACT_RELU, QUICK>(a, b); break;
        case GPTQ_ACT_SILU: gate_of<GPTQ_ACT_SILU, QUICK>(a, b); break;
        case GPTQ_ACT_GELU: gate_of<GPTQ_ACT_GELU, QUICK>(a, b); break;
        case GPTQ_ACT_GELU_TANH: gate_of<GPTQ_ACT_GELU_TANH, QUICK>(a, b); break;
        default: gate_of<GPTQ_ACT_NONE, QUICK>(a, b); break;
    }
}
// (a, b) <- dy times (d act(a) b / da, d act(a) b / db).
template <int ACT, bool QUICK, int N>
__device__ __forceinline__ void gated_grads_of(float (&a)[N], float (&b)[N], const float (&dy)[N]) {
#pragma unroll
    for (int v = 0; v < N; ++v) {
        float y;
        const float k = slope<ACT, QUICK>(a[v], y);
        a[v] = dy[v] * b[v] * k;
        b[v] = dy[v] * y;
    }
}
template <bool QUICK, int N>
__device__ __forceinline__ void gated_grads(float (&a)[N], float (&b)[N], const float (&dy)[N], int act) {
    switch (act) {
        case GPTQ_ACT_RELU: gated_grads_of<GPTQ_ACT_RELU, QUICK>(a, b, dy); break;
        case GPTQ_ACT_SILU: gated_grads_of<GPTQ_ACT_SILU, QUICK>(a, b, dy); break;
        case GPTQ_ACT_GELU: gated_grads_of<GPTQ_ACT_GELU, QUICK>(a, b, dy); break;
        case GPTQ_ACT_GELU_TANH: gated_grads_of<GPTQ_ACT_GELU_TANH, QUICK>(a, b, dy); break;
        default: gated_grads_of<GPTQ_ACT_NONE, QUICK>(a, b, dy); break;
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

// The same of two matrices' sums.
template <int DT, int EPI>
__device__ __forceinline__ void finish_two(const LinArgs& l, int tok, int r, float a, float b) {
    if (l.bias) a += l.bias[r];
    if (l.bias2) b += l.bias2[r];
    if constexpr (EPI == EPI_GATED) {
        float y[1] = {a};
        const float up[1] = {b};
        gate_all<DT != GPTQ_F32>(y, up, l.act);
        store_one<DT>(l.Y, (int64_t)tok * l.ldy + r, y[0]);
    } else {
        float da[1] = {a}, db[1] = {b};
        const float dy[1] = {load_one<DT>(l.R, (int64_t)tok * l.ldr + r)};
        gated_grads<DT != GPTQ_F32>(da, db, dy, l.act);
        float* y = (float*)l.Y + (int64_t)tok * l.ldy + r;
        y[0] = da[0];
        y[l.side] = db[0];
    }
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
    // The same as levels, q - 8, exact in bf16.
    __device__ static u32v4 levels(uint32_t w) {
        const uint32_t even = nibble_bytes(w, false), odd = nibble_bytes(w, true);
        return u32v4{decode_pair<0, 2>(even, 1.0f, -8.0f, 1.0f, -8.0f), decode_pair<0, 2>(odd, 1.0f, -8.0f, 1.0f, -8.0f),
                     decode_pair<1, 3>(even, 1.0f, -8.0f, 1.0f, -8.0f), decode_pair<1, 3>(odd, 1.0f, -8.0f, 1.0f, -8.0f)};
    }
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
    // q - 1.5: both bytes of its bf16 looked up by q, the high ones 4 on.
    __device__ static uint32_t level_pair(uint32_t x) {
        const uint32_t q = x & 0x00030003u;
        return __builtin_amdgcn_perm(0x3f3fbfbfu, 0xc00000c0u, q | q << 8 | 0x04000400u);
    }
    __device__ static u32v4 levels(uint32_t w) {
        const uint32_t x = __builtin_amdgcn_perm(0u, w, 0x0c010c00u);
        return u32v4{level_pair(x), level_pair(x >> 2), level_pair(x >> 4), level_pair(x >> 6)};
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
template <int DT, int BITS, int RT, int TT, int NW, int PD, int EPI>
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
        const int64_t row = min(matrix_row<EPI>(row0 + 16 * i + c), a.rows - 1);
        const bool second = EPI != EPI_LINEAR && i % 2;
        cp[i] = (second ? a.codes2 : a.codes) + row * a.G * Code<BITS>::kBytes;
        sp[i] = (second ? a.scale2 : a.scale) + row * a.G;
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
                for (int i = 0; i < RT; ++i)
                    code[i] = kLevels<DT, EPI> ? Code<BITS>::levels(w[p].w[i][j]) : Code<BITS>::operand(w[p].w[i][j]);
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) {
                    u32v4 t[NT];
                    raw_terms<DT>(x[p][j][tt].a, t);
                    f32v4 start = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (!kLevels<DT, EPI>)
#pragma unroll
                        for (int k = 0; k < NT; ++k) start = mfma16(t[k], offset, start);
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        f32v4 d = start;
                        if constexpr (kLevels<DT, EPI>)  // from the small terms up
#pragma unroll
                            for (int k = NT - 1; k >= 0; --k) d = mfma16(t[k], code[i], d);
                        else
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
    if constexpr (EPI != EPI_LINEAR) {
        // Outputs of two tiles of sums each: 16 rows of both matrices.
        for (int u = wave; u < RT / 2 * TT * 4; u += NW) {
            const int at = (u >> 2) / TT * 2, tt = (u >> 2) % TT, v0 = (at * TT + tt) * 4 + (u & 3);
            float z0 = 0.0f, z1 = 0.0f;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                z0 += red[k][v0][lane];
                z1 += red[k][v0 + TT * 4][lane];
            }
            const int tok = tok0 + tt * 16 + 4 * h + (u & 3), v = row0 + at * 16 + c, r = matrix_row<EPI>(v);
            if (tok >= a.t || r >= a.rows) continue;
            if (a.part) {
                float* p = a.part + ((int64_t)blockIdx.z * a.t + tok) * sums_of(EPI, a.rows) + v;
                p[0] = z0;
                p[16] = z1;
            } else {
                finish_two<DT, EPI>(a, tok, r, z0, z1);
            }
        }
        return;
    }
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

template <int DT, int BITS, int RT, int TT, int EPI>
__global__ __launch_bounds__(kTileWaves * 64) void linear_tile_kernel(LinArgs a) {
    constexpr int NT = kTerms<DT>;
    constexpr int KC = (NT == 3 ? 4 : 8) / TT;       // quads of a chunk
    constexpr int F = KC * 4 * TT;                   // 16-token operands of a chunk (one group each)
    constexpr int FT = F / kTileWaves;               // .. that a wave prepares
    constexpr int PD = KC < 2 ? 1 : 2;               // quads of codes in flight; KC is a multiple of it
    __shared__ u32v4 xs[2][F][NT][64];
    constexpr bool STARTS = NT > 1 && !kLevels<DT, EPI>;  // start values are kept beside the operands
    __shared__ f32v4 start[2][STARTS ? F : 1][4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int row0 = (blockIdx.x * kTileWaves + wave) * 16 * RT, tok0 = blockIdx.y * 16 * TT;
    const int all = (a.G + 3) >> 2;
    const int first = (int)((int64_t)all * blockIdx.z / gridDim.z), end = (int)((int64_t)all * (blockIdx.z + 1) / gridDim.z);
    const uint8_t* cp[RT];
    const float* sp[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int64_t row = min(matrix_row<EPI>(row0 + 16 * i + c), a.rows - 1);
        const bool second = EPI != EPI_LINEAR && i % 2;
        cp[i] = (second ? a.codes2 : a.codes) + row * a.G * Code<BITS>::kBytes;
        sp[i] = (second ? a.scale2 : a.scale) + row * a.G;
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
            if constexpr (STARTS) {
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
                for (int i = 0; i < RT; ++i)
                    code[i] = kLevels<DT, EPI> ? Code<BITS>::levels(now[i][j]) : Code<BITS>::operand(now[i][j]);
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) {
                    const int f = (k * 4 + j) * TT + tt;
                    u32v4 x[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) x[n] = xs[buf][f][n][lane];
                    f32v4 d0 = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (NT == 1)
                        d0 = mfma16(x[0], offset, d0);
                    else if constexpr (STARTS)
                        d0 = start[buf][f][h];
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        f32v4 d = d0;
                        if constexpr (kLevels<DT, EPI>)
#pragma unroll
                            for (int n = NT - 1; n >= 0; --n) d = mfma16(x[n], code[i], d);
                        else
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
    if constexpr (EPI != EPI_LINEAR) {
#pragma unroll
        for (int i = 0; i < RT; i += 2)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tok = tok0 + tt * 16 + 4 * h + r, v = row0 + 16 * i + c, row = matrix_row<EPI>(v);
                    if (tok >= a.t || row >= a.rows) continue;
                    if (a.part) {
                        float* p = a.part + ((int64_t)blockIdx.z * a.t + tok) * sums_of(EPI, a.rows) + v;
                        p[0] = acc[i][tt][r];
                        p[16] = acc[i + 1][tt][r];
                    } else {
                        finish_two<DT, EPI>(a, tok, row, acc[i][tt][r], acc[i + 1][tt][r]);
                    }
                }
        return;
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
template <int DT, int EPI>
__global__ __launch_bounds__(256) void linear_join_two_kernel(LinArgs a, int splits) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.t * a.rows) return;
    const int tok = (int)(i / a.rows), r = (int)(i - (int64_t)tok * a.rows);
    const int64_t wide = sums_of(EPI, a.rows);
    const float* p = a.part + tok * wide + (r >> 4) * 32 + (r & 15);
    float z0 = 0.0f, z1 = 0.0f;
    for (int s = 0; s < splits; ++s, p += a.t * wide) {
        z0 += p[0];
        z1 += p[16];
    }
    finish_two<DT, EPI>(a, tok, r, z0, z1);
}

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

template <int DT, int BITS, int EPI>
static LinKernel codes_kernel(const CodesPlan& c) {
    if constexpr (EPI == EPI_LINEAR)
        if (c.waves == 16) return linear_codes_kernel<DT, BITS, 1, 1, 16, 2, EPI>;
    if (c.waves == 8) return linear_codes_kernel<DT, BITS, 2, 1, 8, 2, EPI>;
    return c.tt == 2 ? linear_tile_kernel<DT, BITS, 2, 2, EPI> : linear_tile_kernel<DT, BITS, 2, 4, EPI>;
}

}  // namespace gptq
