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
#include "common.hpp"
#include "linear_dense.hpp"

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
    const LinArgs a{X,  ldx,      codes,     scale,  bias, residual, ldr,     Y,       ldy,
                    (int)t, (int)rows, (int)G, act, nullptr, nullptr, nullptr, nullptr, 0};
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
        dtype == GPTQ_F32    ? (four ? codes_kernel<GPTQ_F32, 4, EPI_LINEAR>(ct) : codes_kernel<GPTQ_F32, 2, EPI_LINEAR>(ct))
        : dtype == GPTQ_BF16 ? (four ? codes_kernel<GPTQ_BF16, 4, EPI_LINEAR>(ct) : codes_kernel<GPTQ_BF16, 2, EPI_LINEAR>(ct))
                             : (four ? codes_kernel<GPTQ_F16, 4, EPI_LINEAR>(ct) : codes_kernel<GPTQ_F16, 2, EPI_LINEAR>(ct));
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
