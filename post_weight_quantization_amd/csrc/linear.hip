// linear.hip -- Y = act(X W^T + bias) + residual from the sweeps' codes on gfx950.
//
// W[r][j] = (q[r][j] - z) s[r][j / 32], z = 8 for q4tp's nibbles and 1.5 for q2tp's 2-bit codes,
// so a group of 32 columns adds s (sum_j q_j x_j - z sum_j x_j) to an output.  One 16x16x32 MFMA is
// one group: A = 16 tokens of X, B = the codes of 16 rows as whole numbers (codes16.hpp), and
// the result, exact up to f32 sums, is scaled by the lane's own s (D's column is the row of W)
// into the accumulator.  z and the operand's offset come out through the start value of D: X times
// a constant operand.  f16 and f32 X enter as two and three exact bf16 terms.
//
// linear_codes_kernel: a workgroup owns 16 rows of W and 16 TT tokens; its waves take quads of
// four groups in turn and their sums are joined in LDS, where the epilogue runs.  Per quad a lane
// loads 16 bytes (q4tp), one group of its row; a 4 x 4 transpose over the lane's quarter of the
// wave (four permlane swaps) hands each quarter its eight columns of every group.
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
};

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == GPTQ_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if constexpr (ACT == GPTQ_ACT_SILU) return z / (1.0f + expf(-z));
    if constexpr (ACT == GPTQ_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    if constexpr (ACT == GPTQ_ACT_GELU_TANH)
        return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
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
        return u32v4{((x << 5) & 0x00600060u) | 0x40804080u, ((x << 3) & 0x00600060u) | 0x40804080u,
                     ((x << 1) & 0x00600060u) | 0x40804080u, ((x >> 1) & 0x00600060u) | 0x40804080u};
    }
};

template <int DT, int BITS, int TT, int NW>
__global__ __launch_bounds__(NW * 64) void linear_codes_kernel(LinArgs a) {
    constexpr int NT = kTerms<DT>;
    __shared__ float red[NW][TT * 4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, h = lane >> 4;
    const int row0 = blockIdx.x * 16, tok0 = blockIdx.y * 16 * TT;
    const int64_t row = min(row0 + c, a.rows - 1);
    const uint8_t* cp = a.codes + row * a.G * Code<BITS>::kBytes;
    const float* sp = a.scale + row * a.G;
    int64_t xo[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) xo[tt] = (int64_t)min(tok0 + tt * 16 + c, a.t - 1) * a.ldx + 8 * h;
    f32v4 acc[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) acc[tt] = f32v4{0.f, 0.f, 0.f, 0.f};
    const u32v4 offset = {Code<BITS>::kOffset, Code<BITS>::kOffset, Code<BITS>::kOffset, Code<BITS>::kOffset};

    const int quads = (a.G + 3) >> 2;
    for (int q = wave; q < quads; q += NW) {
        uint32_t w[4];
        Code<BITS>::load(cp + (int64_t)min(4 * q + h, a.G - 1) * Code<BITS>::kBytes, w);
        float s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = sp[min(4 * q + j, a.G - 1)];
        transpose_quarters(w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (4 * q + j >= a.G) break;  // the same in every lane
            const u32v4 b = Code<BITS>::operand(w[j]);
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                u32v4 x[NT];
                load_terms<DT, true>(a.X, xo[tt] + 32 * (4 * q + j), x);
                f32v4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < NT; ++k) d = mfma16(x[k], offset, d);
#pragma unroll
                for (int k = 0; k < NT; ++k) d = mfma16(x[k], b, d);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[tt][r] = fmaf(s[j], d[r], acc[tt][r]);
            }
        }
    }
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][tt * 4 + r][lane] = acc[tt][r];
    __syncthreads();
    for (int i = wave; i < TT * 4; i += NW) {
        float z = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) z += red[k][i][lane];
        const int tok = tok0 + (i >> 2) * 16 + 4 * h + (i & 3), r = row0 + c;
        if (tok < a.t && r < a.rows) {
            float y[1] = {a.bias ? z + a.bias[r] : z};
            activate_all(y, a.act);
            if (a.R) y[0] += load_one<DT>(a.R, (int64_t)tok * a.ldr + r);
            store_one<DT>(a.Y, (int64_t)tok * a.ldy + r, y[0]);
        }
    }
}

}  // namespace gptq

#include "linear_dense.hpp"

namespace gptq {

typedef void (*LinKernel)(LinArgs);
constexpr int kLinWaves = 8;

template <int DT, int BITS>
static LinKernel codes_kernel(int tt) {
    return tt == 1 ? linear_codes_kernel<DT, BITS, 1, kLinWaves>
           : tt == 2 ? linear_codes_kernel<DT, BITS, 2, kLinWaves>
                     : linear_codes_kernel<DT, BITS, 4, kLinWaves>;
}

}  // namespace gptq

using namespace gptq;

static bool linear_sizes_ok(int dtype, int64_t t, int64_t rows, int64_t n) {
    return dtype_size(dtype) && t >= 0 && t <= (1 << 24) && rows >= 1 && rows <= (1 << 24) && n >= 32 &&
           n <= (1 << 20) && n % 32 == 0;
}

// Many tokens in a 16-bit type run on decoded weights.
static bool linear_dense(int dtype, int64_t t) { return dtype != GPTQ_F32 && t > 128; }
static int64_t dense_ld(int64_t n) { return round_up(n, kTileK); }
// Workspace of the dense product: the arrival counts, the rows' powers of two, the weights (whole tiles
// of rows), the pieces' sums.
struct DenseSpace {
    size_t power, weights, part, bytes;
};
static DenseSpace dense_space(int64_t t, int64_t rows, int64_t n) {
    const DensePlan p = dense_plan(t, rows, n);
    DenseSpace s;
    s.power = align256(sizeof(uint32_t) * kCUs);
    s.weights = s.power + align256(sizeof(float) * (size_t)rows);
    s.part = s.weights + align256(2 * (size_t)round_up(rows, kTileR) * (size_t)dense_ld(n));
    s.bytes = s.part + sizeof(float) * (size_t)((p.tiles - p.whole) * p.splits) * (kTileT * kTileR);
    return s;
}

extern "C" size_t gptq_linear_workspace_size(int dtype, int64_t t, int64_t rows, int64_t n) {
    if (!linear_sizes_ok(dtype, t, rows, n) || !linear_dense(dtype, t)) return 0;
    return dense_space(t, rows, n).bytes;
}

template <int DT>
static int linear_dense_run(const LinArgs& l, bool four, int64_t n, void* workspace, hipStream_t st) {
    const DenseSpace sp = dense_space(l.t, l.rows, n);
    const DensePlan p = dense_plan(l.t, l.rows, n);
    char* ws = (char*)workspace;
    const DenseArgs d{l, (uint16_t*)(ws + sp.weights), (float*)(ws + sp.power), (int)dense_ld(n), (int)n,
                      (int)p.tiles_r, (int)p.tiles, (int)p.whole, (int)p.splits, (float*)(ws + sp.part), (uint32_t*)ws};
    const int64_t ldw = d.ldw, cb = four ? n / 2 : n / 4, cut = (p.tiles - p.whole) * p.splits;
    const int64_t sums = cut * kTileT * kTileR;
    uint16_t* W = (uint16_t*)d.W;
    float* power = (float*)d.power;
    {
        ProfScope ps(FAM_LINEAR, st, 0.0, (double)l.rows * (cb + 4 * l.G + 2 * ldw));
        GPTQ_LAUNCH(st, "linear_decode",
                    (four ? decode_kernel<DT, 4><<<(unsigned)l.rows, 256, 0, st>>>(l, W, power, d.ldw, d.arrived)
                          : decode_kernel<DT, 2><<<(unsigned)l.rows, 256, 0, st>>>(l, W, power, d.ldw, d.arrived)),
                    rd(l.codes, cb, l.rows, cb, 1), rd(l.scale, l.G, l.rows, l.G), wr(W, ldw, l.rows, ldw, 2),
                    wr(power, l.rows, DT == GPTQ_F16 ? 1 : 0, l.rows), wr(d.arrived, kCUs, 1, kCUs));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    ProfScope ps(FAM_LINEAR, st, 2.0 * (double)l.t * l.rows * n, 0.0);
    GPTQ_LAUNCH(st, "linear_dense",
                (dense_kernel<DT><<<(unsigned)(p.whole + cut), kDenseWaves * 64, 0, st>>>(d)),
                rd(l.X, l.ldx, l.t, n, 2), rd(W, ldw, round_up(l.rows, kTileR), ldw, 2),
                rd(power, l.rows, DT == GPTQ_F16 ? 1 : 0, l.rows),
                rd(l.bias ? l.bias : l.scale, l.rows, l.bias ? 1 : 0, l.rows),
                rd(l.R ? l.R : (const void*)l.scale, l.ldr, l.R ? l.t : 0, l.rows, 2), wr(l.Y, l.ldy, l.t, l.rows, 2),
                wr(d.part, sums, cut ? 1 : 0, sums), wr(d.arrived, kCUs, cut ? 1 : 0, kCUs));
    return GPTQ_OK;
}

extern "C" int gptq_linear(const void* X, int64_t ldx, int dtype, int64_t t, int codec,
                           const uint8_t* codes, const float* scale, int64_t rows, int64_t n,
                           const float* bias, int act, const void* residual, int64_t ldr, void* Y,
                           int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
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
    const size_t need = gptq_linear_workspace_size(dtype, t, rows, n);
    if (need) {
        if (!workspace || workspace_bytes < need) return GPTQ_EWORKSPACE;
        if ((uintptr_t)workspace & 255u) return GPTQ_EINVAL;
    }
    CheckScope check;
    if (need) check_buffer(workspace, workspace_bytes, "workspace");
    const int64_t G = n / 32, cb = codec == GPTQ_CODEC_Q4TP ? n / 2 : n / 4;
    check_buffer(X, (size_t)es * (size_t)((t - 1) * ldx + n), "X");
    check_buffer(codes, (size_t)(rows * cb), "codes");
    check_buffer(scale, sizeof(float) * (size_t)(rows * G), "scale");
    if (bias) check_buffer(bias, sizeof(float) * (size_t)rows, "bias");
    if (residual) check_buffer(residual, (size_t)es * (size_t)((t - 1) * ldr + rows), "residual");
    check_buffer(Y, (size_t)es * (size_t)((t - 1) * ldy + rows), "Y");
    hipStream_t st = (hipStream_t)stream;
    const LinArgs a{X, ldx, codes, scale, bias, residual, ldr, Y, ldy, (int)t, (int)rows, (int)G, act};
    if (need) {
        const bool q4 = codec == GPTQ_CODEC_Q4TP;
        const int rc = dtype == GPTQ_BF16 ? linear_dense_run<GPTQ_BF16>(a, q4, n, workspace, st)
                                          : linear_dense_run<GPTQ_F16>(a, q4, n, workspace, st);
        if (rc != GPTQ_OK) return rc;
        if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
        return check.finish();
    }
    const int tt = t <= 16 ? 1 : t <= 32 ? 2 : 4;
    const bool four = codec == GPTQ_CODEC_Q4TP;
    const LinKernel k =
        dtype == GPTQ_F32    ? (four ? codes_kernel<GPTQ_F32, 4>(tt) : codes_kernel<GPTQ_F32, 2>(tt))
        : dtype == GPTQ_BF16 ? (four ? codes_kernel<GPTQ_BF16, 4>(tt) : codes_kernel<GPTQ_BF16, 2>(tt))
                             : (four ? codes_kernel<GPTQ_F16, 4>(tt) : codes_kernel<GPTQ_F16, 2>(tt));
    // Grid y is limited to 65535; 2^24 tokens are launched in slices of 2^21.
    for (int64_t t0 = 0; t0 < t; t0 += 1 << 21) {
        LinArgs b = a;
        b.t = (int)(t - t0 < (1 << 21) ? t - t0 : (1 << 21));
        b.X = (const char*)X + t0 * ldx * es;
        b.Y = (char*)Y + t0 * ldy * es;
        if (residual) b.R = (const char*)residual + t0 * ldr * es;
        const dim3 grid((unsigned)((rows + 15) / 16), (unsigned)((b.t + 16 * tt - 1) / (16 * tt)));
        ProfScope ps(FAM_LINEAR, st, 2.0 * (double)b.t * rows * n, (double)rows * (cb + 4 * G));
        GPTQ_LAUNCH(st, "linear_codes", (k<<<grid, kLinWaves * 64, 0, st>>>(b)), rd(b.X, ldx, b.t, n, es),
                    rd(codes, cb, rows, cb, 1), rd(scale, G, rows, G),
                    rd(bias ? (const void*)bias : (const void*)scale, rows, bias ? 1 : 0, rows),
                    rd(residual ? b.R : (const void*)scale, ldr, residual ? b.t : 0, rows, es),
                    wr(b.Y, ldy, b.t, rows, es));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}
