// gated.hip -- the gated feed-forward block, Y = act(X Wg^T + bg) (X Wu^T + bu), from the sweeps' codes on
// gfx950, and the gradient of X.
//
// Both products run as one whose rows are the two matrices' in turns of 16 (linear_codes.hpp, sums_of): the sums
// of an output meet in one lane, so that X is read once and only Y is written.  Few tokens, and f32, run on
// the codes as gptq_linear does; many in a 16-bit type on weights decoded to f16 (dense16.hpp), for f16 in two terms.
//
// The gradient makes both sums again, from X: with them in registers the epilogue turns dY into the gradients of
// the two sums, and those are the operand of one more product, over the rows of both matrices (backward.hpp, or
// dense16.hpp with the weights turned).  Nothing of the forward pass has to be kept for it but X.
#include "../../include/gptq_check.h"
#include "backward.hpp"
#include "check.hpp"
#include "dense16.hpp"

namespace gptq {

// A caller's type: with GPTQ_EXACT_WEIGHTS no size is multiplied on decoded weights.
static int plain_type(int type) { return type & ~GPTQ_EXACT_WEIGHTS; }
// Many tokens in a 16-bit type run on decoded weights, where there is enough to multiply for three launches, in the
// gradient seven.  Measured (us, codes / decoded; tokens of rows x n, products of both matrices):
//   bf16      1000 of 2048 x 2048 (8e9) 39 / 47, 2500 of 2500 x 512 (6e9) 54 / 49, 200 of 5120 x 17408 (36e9) 183 / 223
//   gradient  139 / 120, 228 / 128, 601 / 500; 200 of 4096 x 4096 (7e9) 130 / 132, 512 of 4096 x 1024 (4e9) 88 / 111; 100 of
//             5120 x 17408 356 / 485
//   f16, whose decoded weights are two terms: 512 of 5120 x 17408 (91e9) 477 / 524, of 5120 x 5120 174 / 168; 450 of 4096 x
//             4096 (15e9) 85 / 103; 1200 of 2048 x 2048 (10e9) 85 / 68, 600 of 2048 x 4096 (10e9) 75 / 77, 800 of 4096 x 1024 52 / 63
//   gradient  300 of 5120 x 17408 852 / 964, 400 1116 / 990; 350 of 4096 x 4096 205 / 229, 390 241 / 236; 800 of 2048 x 2048
//             (7e9) 138 / 126, 2600 of 2500 x 512 (7e9) 229 / 126
static bool gated_dense(int type, int64_t t, int64_t rows, int64_t n, bool back) {
    if ((type != GPTQ_BF16 && type != GPTQ_F16) || rows > (1 << 20)) return false;
    const int64_t products = 2 * t * rows * n;
    if (back) return t > (type == GPTQ_BF16 ? 160 : 384) && products > 6500000000;
    return t > (type == GPTQ_BF16 ? 256 : 512) && products > 10000000000;
}
static bool gated_sizes_ok(int dtype, int64_t t, int64_t rows, int64_t n) {
    return dtype_size(dtype) && t >= 0 && t <= (1 << 24) && rows >= 1 && rows <= (1 << 22) && t * rows <= ((int64_t)1 << 38) &&
           n >= 32 && n <= (1 << 20) && n % 32 == 0 && t * n <= ((int64_t)1 << 38);
}

// The products on decoded weights of `t` tokens at once: the sums, and (backward) the gradients times both matrices.  K as
// the kernel steps through it, whole tiles of each of `terms`.
static DensePlan sums_plan(int terms, int64_t t, int64_t rows, int64_t n) {
    return dense16_plan(t, sums_of(EPI_GATED, rows), terms * round_up(n, kTileK));
}
static DensePlan grad_plan(int terms, int64_t t, int64_t rows, int64_t n) { return dense16_plan(t, n, terms * 2 * round_up(rows, kTileK)); }

// Workspace on decoded weights: X's powers and largest magnitudes, dY's, the weights' powers and bounds; X', W',
// (backward) the gradients of the sums and W' turned, pieces.
struct GatedSpace {
    int64_t ldx, ldw, ldd, slice, side;
    size_t top_x, grad, power, bound, row_bound, X, W, D, T, part, bytes;
};
static GatedSpace gated_space(int type, int64_t t, int64_t rows, int64_t n, bool back) {
    GatedSpace s;
    const int terms = block_terms(type);
    s.ldx = round_up(n, kTileK);
    s.ldw = terms * s.ldx;
    s.side = round_up(rows, kTileK);
    s.ldd = terms * 2 * s.side;
    s.slice = t < kTokens16 ? t : kTokens16;
    const size_t tokens = align256(4 * (size_t)s.slice);
    const int64_t sums = sums_of(EPI_GATED, rows);
    s.top_x = tokens;
    s.grad = s.top_x + tokens;
    s.power = s.grad + tokens;
    s.bound = s.power + align256(4 * (size_t)sums);
    s.row_bound = s.bound + align256(sizeof(GradBound));
    s.X = s.row_bound + (back ? align256(8 * (size_t)rows) : 0);
    s.W = s.X + align256(2 * (size_t)s.slice * (size_t)s.ldx);
    s.D = s.W + align256(2 * (size_t)round_up(sums, kTileR) * (size_t)s.ldw);
    s.T = s.D + (back ? align256(2 * (size_t)s.slice * (size_t)s.ldd) : 0);
    s.part = s.T + (back ? align256(4 * (size_t)round_up(n, kTileR) * (size_t)s.side) : 0);
    s.bytes = s.part;
    for (int64_t k : {s.slice, t % s.slice}) {
        if (!k) continue;
        for (int product = 0; product < (back ? 2 : 1); ++product) {
            const DensePlan p = product ? grad_plan(terms, k, rows, n) : sums_plan(terms, k, rows, n);
            const size_t b = s.part + sizeof(float) * (size_t)((p.tiles - p.whole) * p.splits) * (kTileT * kTileR);
            if (b > s.bytes) s.bytes = b;
        }
    }
    return s;
}

// Workspace on codes, kTokens16 tokens at a time: the pieces' sums, then (backward) the gradients of the sums in
// f32 and the pieces of their product.
static int64_t grad_side(int64_t rows) { return round_up(rows, 8); }
struct GatedCodes {
    CodesPlan sums;
    BackPlan back;
    size_t D, part, bytes;
};
static GatedCodes gated_codes(int64_t t, int64_t rows, int64_t n, bool back) {
    GatedCodes g{};
    const int64_t sums = sums_of(EPI_GATED, rows);
    g.sums = codes_plan(t, sums, n);
    // Two matrices' rows are tiles of 32 at least, on which 8 waves are never slower than 16: one token of 8192 x 2048 8.7
    // against 9.7 us, 4096 x 4096 alike.
    if (g.sums.waves == 16) g.sums.waves = 8;
    g.D = g.sums.splits > 1 ? align256(sizeof(float) * (size_t)g.sums.splits * (size_t)t * (size_t)sums) : 0;
    g.part = g.bytes = g.D;
    if (back) {
        g.back = back_plan(t, rows, 2, n);
        g.part = g.D + align256(2 * sizeof(float) * (size_t)t * (size_t)grad_side(rows));
        g.bytes = g.part + back_part_bytes(g.back, t, n);
    }
    return g;
}
static size_t gated_bytes(int type, int64_t t, int64_t rows, int64_t n, bool back) {
    if (!gated_sizes_ok(plain_type(type), t, rows, n) || t == 0) return 0;
    if (gated_dense(type, t, rows, n, back)) return gated_space(type, t, rows, n, back).bytes;
    size_t most = 0;
    for (int64_t k : {t < kTokens16 ? t : kTokens16, t % kTokens16})
        if (k) {
            const size_t b = gated_codes(k, rows, n, back).bytes;
            if (b > most) most = b;
        }
    return most;
}

// The two matrices' sums on codes, and what EPI makes of them.
template <int DT, int EPI>
static int sums_run(LinArgs a, const CodesPlan& c, int bits, int64_t n, hipStream_t st) {
    const LinKernel k = bits == 4 ? codes_kernel<DT, 4, EPI>(c) : codes_kernel<DT, 2, EPI>(c);
    const int64_t es = dtype_size(DT), sums = sums_of(EPI, a.rows), cb = (int64_t)a.G * 4 * bits;
    const int64_t tile = 32 * (c.waves ? 1 : kTileWaves);
    const dim3 grid((unsigned)((sums + tile - 1) / tile), (unsigned)((a.t + 16 * c.tt - 1) / (16 * c.tt)), (unsigned)c.splits);
    const Span y = EPI == EPI_GATED ? wr(a.Y, a.ldy, a.t, a.rows, (int)es) : wr(a.Y, a.ldy, a.t, a.side + a.rows);
    auto bias = [&](const float* p) { return rd(p ? p : a.scale, a.rows, p ? 1 : 0, a.rows); };
    const Span dy = rd(a.R ? a.R : (const void*)a.scale, a.ldr, a.R ? a.t : 0, a.rows, (int)es);
    ProfScope ps(FAM_LINEAR, st, 4.0 * (double)a.t * a.rows * n, 2.0 * (double)a.rows * (cb + 4 * a.G));
    GPTQ_LAUNCH(st, "gated_codes", (k<<<grid, (c.waves ? c.waves : kTileWaves) * 64, 0, st>>>(a)), rd(a.X, a.ldx, a.t, n, (int)es),
                rd(a.codes, cb, a.rows, cb, 1), rd(a.scale, a.G, a.rows, a.G), rd(a.codes2, cb, a.rows, cb, 1),
                rd(a.scale2, a.G, a.rows, a.G), bias(a.bias), bias(a.bias2), dy,
                a.part ? wr(a.part, sums, (int64_t)a.t * c.splits, sums) : y);
    if (a.part)
        GPTQ_LAUNCH(st, "gated_join",
                    (linear_join_two_kernel<DT, EPI><<<(unsigned)(((int64_t)a.t * a.rows + 255) / 256), 256, 0, st>>>(a, c.splits)),
                    rd(a.part, sums, (int64_t)a.t * c.splits, sums), bias(a.bias), bias(a.bias2), dy, y);
    return GPTQ_OK;
}

// One pass: Y, or (dY given) dX.
struct GatedCall {
    const void* X;
    int64_t ldx;
    int type;
    int64_t t;
    int bits;
    const gptq_weights* w[2];
    int64_t rows, n;
    int act;
    const void* dY;
    int64_t ldd;
    void* Y;  // or dX
    int64_t ldy;
    void* workspace;
};

template <int DT>
static int gated_codes_run(const GatedCall& g, hipStream_t st) {
    const int64_t es = dtype_size(DT);
    for (int64_t t0 = 0; t0 < g.t; t0 += kTokens16) {
        const int64_t k = g.t - t0 < kTokens16 ? g.t - t0 : kTokens16;
        const GatedCodes p = gated_codes(k, g.rows, g.n, g.dY != nullptr);
        char* ws = (char*)g.workspace;
        const int64_t side = grad_side(g.rows);
        float* D = (float*)(ws + p.D);
        char* y = (char*)g.Y + t0 * g.ldy * es;
        LinArgs a{(const char*)g.X + t0 * g.ldx * es, g.ldx, g.w[0]->codes, g.w[0]->scale, g.w[0]->bias,
                  g.dY ? (const char*)g.dY + t0 * g.ldd * es : nullptr, g.ldd, g.dY ? (void*)D : (void*)y, g.dY ? 2 * side : g.ldy,
                  (int)k, (int)g.rows, (int)(g.n / 32), g.act, p.sums.splits > 1 ? (float*)ws : nullptr, g.w[1]->codes,
                  g.w[1]->scale, g.w[1]->bias, (int)side};
        const int rc = g.dY ? sums_run<DT, EPI_GRAD>(a, p.sums, g.bits, g.n, st) : sums_run<DT, EPI_GATED>(a, p.sums, g.bits, g.n, st);
        if (rc != GPTQ_OK) return rc;
        if (!g.dY) continue;
        if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
        const BackArgs b{D, 2 * side, (int)side, 2, (int)g.rows, (int)(g.n / 32), (int)g.n, {g.w[0]->codes, g.w[1]->codes},
                         {g.w[0]->scale, g.w[1]->scale}, (int)k, y, g.ldy, (float*)(ws + p.part)};
        const int rb = back_run(b, p.back, GPTQ_F32, DT, g.bits, st);
        if (rb != GPTQ_OK) return rb;
    }
    return GPTQ_OK;
}

template <int DT>
static int gated_dense_run(const GatedCall& g, hipStream_t st) {
    const bool back = g.dY != nullptr;
    const GatedSpace s = gated_space(DT, g.t, g.rows, g.n, back);
    constexpr int terms = block_terms(DT);
    const int64_t G = g.n / 32, cb = G * 4 * g.bits, sums = sums_of(EPI_GATED, g.rows);
    char* ws = (char*)g.workspace;
    float *token = (float*)ws, *top_x = (float*)(ws + s.top_x), *grad = (float*)(ws + s.grad), *power = (float*)(ws + s.power);
    GradBound* bound = (GradBound*)(ws + s.bound);
    f32v2* row_bound = back ? (f32v2*)(ws + s.row_bound) : nullptr;
    uint16_t *X = (uint16_t*)(ws + s.X), *W = (uint16_t*)(ws + s.W), *D = (uint16_t*)(ws + s.D), *T = (uint16_t*)(ws + s.T);
    float* part = (float*)(ws + s.part);
    LinArgs w{};
    w.codes = g.w[0]->codes;
    w.scale = g.w[0]->scale;
    w.bias = g.w[0]->bias;
    w.codes2 = g.w[1]->codes;
    w.scale2 = g.w[1]->scale;
    w.bias2 = g.w[1]->bias;
    w.G = (int)G;
    w.act = g.act;
    auto matrix = [&](int m) { return rd(g.w[m]->codes, cb, g.rows, cb, 1); };
    auto scales = [&](int m) { return rd(g.w[m]->scale, G, g.rows, G); };
    auto biases = [&](int m) { return rd(g.w[m]->bias ? g.w[m]->bias : g.w[m]->scale, g.rows, g.w[m]->bias ? 1 : 0, g.rows); };
    ProfScope ps(FAM_LINEAR, st, (back ? 8.0 : 4.0) * (double)g.t * g.rows * g.n, 0.0);
    for (int64_t t0 = 0; t0 < g.t; t0 += s.slice) {
        const int64_t k = g.t - t0 < s.slice ? g.t - t0 : s.slice;
        const Halve hx{(const char*)g.X + t0 * g.ldx * 2, g.ldx, (int)g.n, nullptr, X, (int)s.ldx, token, top_x, nullptr};
        GPTQ_LAUNCH(st, "gated_halve", (halve_kernel<DT><<<(unsigned)k, 256, 0, st>>>(hx)), rd(hx.X, g.ldx, k, g.n, 2),
                    wr(X, s.ldx, k, s.ldx, 2), wr(token, k, 1, k), wr(top_x, k, 1, k));
        if (t0 == 0) {
            GPTQ_LAUNCH(st, "gated_decode",
                        (g.bits == 4 ? decode_two_kernel<4, terms == 2><<<(unsigned)g.rows, 256, 0, st>>>(w, W, power, (int)s.ldx, row_bound)
                                     : decode_two_kernel<2, terms == 2><<<(unsigned)g.rows, 256, 0, st>>>(w, W, power, (int)s.ldx, row_bound)),
                        matrix(0), matrix(1), scales(0), scales(1), biases(0), biases(1), wr(W, s.ldw, sums, s.ldw, 2),
                        wr(power, sums, 1, sums), wr(ws + s.row_bound, 2 * g.rows, back ? 1 : 0, 2 * g.rows));
            if (back) {
                GPTQ_LAUNCH(st, "gated_bound", (bound_kernel<<<kSlots, 256, 0, st>>>(row_bound, (int)g.rows, bound)),
                            rd(row_bound, 2 * g.rows, 1, 2 * g.rows), wr(bound, 2 * kSlots, 1, 2 * kSlots));
                const Turn turn{{g.w[0]->codes, g.w[1]->codes}, {g.w[0]->scale, g.w[1]->scale}, power, true, (int)g.rows, (int)g.n,
                                (int)s.side, (int)(2 * s.side), T};
                const dim3 grid((unsigned)((g.n + 255) / 256), (unsigned)(s.side / 64), 2);
                GPTQ_LAUNCH(st, "gated_turn", (g.bits == 4 ? turn_kernel<4><<<grid, 256, 0, st>>>(turn) : turn_kernel<2><<<grid, 256, 0, st>>>(turn)),
                            matrix(0), matrix(1), scales(0), scales(1), rd(power, sums, 1, sums), wr(T, 2 * s.side, g.n, 2 * s.side, 2));
            }
            if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
        }
        Dense16 d{};
        d.X = X;
        d.ldx = (int)s.ldx;
        d.t = (int)k;
        d.W = W;
        d.ldw = (int)s.ldw;
        d.power = power;
        d.token = token;
        d.rows = (int)g.rows;
        d.act = g.act;
        d.bias = g.w[0]->bias;
        d.bias2 = g.w[1]->bias;
        d.part = part;
        if (back) {
            const Halve hd{(const char*)g.dY + t0 * g.ldd * 2, g.ldd, (int)g.rows, nullptr, nullptr, 0, grad, top_x, bound};
            GPTQ_LAUNCH(st, "gated_top", (halve_kernel<DT><<<(unsigned)k, 256, 0, st>>>(hd)), rd(hd.X, g.ldd, k, g.rows, 2), rd(top_x, k, 1, k),
                        rd(ws + s.bound, 2 * kSlots, 1, 2 * kSlots), wr(grad, k, 1, k));
            d.dY = hd.X;
            d.ldd = g.ldd;
            d.grad_token = grad;
            d.D = D;
            d.side = (int)s.side;
        } else {
            d.Y = (char*)g.Y + t0 * g.ldy * 2;
            d.ldy = g.ldy;
        }
        const Span tops = rd(grad, k, back ? 1 : 0, k), dy = rd(back ? g.dY : (const void*)X, g.ldd, back ? k : 0, g.rows, 2);
        auto product = [&](bool second) -> int {
            const DensePlan p = second ? grad_plan(terms, k, g.rows, g.n) : sums_plan(terms, k, g.rows, g.n);
            const int64_t cut = (p.tiles - p.whole) * p.splits, all = cut * kTileT * kTileR;
            d.tiles_r = (int)p.tiles_r;
            d.tiles = (int)p.tiles;
            d.whole = (int)p.whole;
            d.splits = (int)p.splits;
            const int mode = second ? DENSE_LAST : back ? DENSE_GRAD : DENSE_GATED;
            void (*const run)(Dense16) = second ? dense16_kernel<DT, DENSE_LAST> : back ? dense16_kernel<DT, DENSE_GRAD> : dense16_kernel<DT, DENSE_GATED>;
            void (*const join)(Dense16) =
                second ? dense16_join_kernel<DT, DENSE_LAST> : back ? dense16_join_kernel<DT, DENSE_GRAD> : dense16_join_kernel<DT, DENSE_GATED>;
            const Span out = mode == DENSE_GRAD ? wr(D, s.ldd, k, s.ldd, 2) : wr(d.Y, d.ldy, k, d.rows, 2);
            GPTQ_LAUNCH(st, "gated_dense16", (run<<<(unsigned)(p.whole + cut), kDenseWaves * 64, 0, st>>>(d)), rd(d.X, d.ldx, k, d.ldx, 2),
                        rd(d.W, d.ldw, round_up(second ? g.n : sums, kTileR), d.ldw, 2), rd(power, sums, 1, sums), rd(token, k, 1, k), tops,
                        biases(0), biases(1), dy, out, wr(part, all, cut ? 1 : 0, all));
            if (cut)
                GPTQ_LAUNCH(st, "gated_dense16_join",
                            (join<<<dim3(kTileT * kTileR / (dense_plain(mode) ? 1024 : 4096), (unsigned)(p.tiles - p.whole)), 256, 0, st>>>(d)),
                            rd(part, all, 1, all), rd(power, sums, 1, sums), rd(token, k, 1, k), tops, biases(0), biases(1), dy, out);
            return launch_status() == GPTQ_OK ? GPTQ_OK : GPTQ_EHIP;
        };
        int rc = product(false);
        if (rc != GPTQ_OK) return rc;
        if (back) {
            d.X = D;
            d.token = grad;
            d.ldx = (int)s.ldd;
            d.W = T;
            d.ldw = (int)(2 * s.side);
            d.rows = (int)g.n;
            d.Y = (char*)g.Y + t0 * g.ldy * 2;
            d.ldy = g.ldy;
            rc = product(true);
            if (rc != GPTQ_OK) return rc;
        }
    }
    return GPTQ_OK;
}

static int gated_call(const GatedCall& g, size_t workspace_bytes, void* stream) {
    const int dtype = plain_type(g.type);
    if (!gated_sizes_ok(dtype, g.t, g.rows, g.n) || g.bits == 0) return GPTQ_EINVAL;
    if (g.act < GPTQ_ACT_NONE || g.act > GPTQ_ACT_GELU_TANH || !g.w[0] || !g.w[1]) return GPTQ_EINVAL;
    if (g.t == 0) return GPTQ_OK;
    const int es = dtype_size(dtype);
    const bool back = g.dY != nullptr;
    const int64_t G = g.n / 32, cb = G * 4 * g.bits, wide = back ? g.n : g.rows, most = (int64_t)1 << 36;
    if (!g.X || !g.Y || g.ldx < g.n || g.ldx > (1 << 22) || g.ldx % (16 / es) || !al16(g.X) || g.ldy < wide || g.ldy > most) return GPTQ_EINVAL;
    if (back && (g.ldd < g.rows || g.ldd > most)) return GPTQ_EINVAL;
    if (((uintptr_t)g.Y | (uintptr_t)g.dY) % (unsigned)es) return GPTQ_EINVAL;
    for (const gptq_weights* w : g.w)
        if (!w->codes || !w->scale || !al16(w->codes) || ((uintptr_t)w->scale | (uintptr_t)w->bias) % 4u) return GPTQ_EINVAL;
    const size_t need = gated_bytes(g.type, g.t, g.rows, g.n, back);
    if (need) {
        if (!g.workspace || workspace_bytes < need) return GPTQ_EWORKSPACE;
        if ((uintptr_t)g.workspace & 255u) return GPTQ_EINVAL;
    }
    auto set = [](const void* p, int64_t bytes) { return RowSet{p, bytes, p && bytes ? 1 : 0, bytes}; };
    const RowSet y{g.Y, g.ldy * es, g.t, wide * es}, ws = set(need ? g.workspace : nullptr, (int64_t)need);
    const RowSet in[] = {RowSet{g.X, g.ldx * es, g.t, g.n * es}, RowSet{g.dY, g.ldd * es, back ? g.t : 0, g.rows * es},
                         set(g.w[0]->codes, g.rows * cb), set(g.w[1]->codes, g.rows * cb), set(g.w[0]->scale, g.rows * G * 4),
                         set(g.w[1]->scale, g.rows * G * 4), set(g.w[0]->bias, g.rows * 4), set(g.w[1]->bias, g.rows * 4)};
    if (rows_meet(y, ws)) return GPTQ_EINVAL;
    for (const RowSet& i : in)
        if (rows_meet(y, i) || rows_meet(ws, i)) return GPTQ_EINVAL;
    CheckScope check;
    if (need) check_buffer(g.workspace, workspace_bytes, "workspace");
    check_buffer(g.X, (size_t)es * (size_t)((g.t - 1) * g.ldx + g.n), "X");
    if (back) check_buffer(g.dY, (size_t)es * (size_t)((g.t - 1) * g.ldd + g.rows), "dY");
    check_buffer(g.Y, (size_t)es * (size_t)((g.t - 1) * g.ldy + wide), "Y");
    for (const gptq_weights* w : g.w) {
        check_buffer(w->codes, (size_t)(g.rows * cb), "codes");
        check_buffer(w->scale, sizeof(float) * (size_t)(g.rows * G), "scale");
        if (w->bias) check_buffer(w->bias, sizeof(float) * (size_t)g.rows, "bias");
    }
    hipStream_t st = (hipStream_t)stream;
    int rc;
    if (gated_dense(g.type, g.t, g.rows, g.n, back))
        rc = dtype == GPTQ_BF16 ? gated_dense_run<GPTQ_BF16>(g, st) : gated_dense_run<GPTQ_F16>(g, st);
    else
        rc = dtype == GPTQ_F32    ? gated_codes_run<GPTQ_F32>(g, st)
             : dtype == GPTQ_BF16 ? gated_codes_run<GPTQ_BF16>(g, st)
                                  : gated_codes_run<GPTQ_F16>(g, st);
    if (rc != GPTQ_OK) return rc;
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}
static int code_bits(int codec) { return codec == GPTQ_CODEC_Q4TP ? 4 : codec == GPTQ_CODEC_Q2TP ? 2 : 0; }

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_check_gated_plan(int type, int64_t t, int64_t rows, int64_t n, int backward, int64_t* plan) {
    if (!plan || !gated_sizes_ok(plain_type(type), t, rows, n) || t == 0) return GPTQ_EINVAL;
    const int64_t k = t < kTokens16 ? t : kTokens16;
    const GatedCodes c = gated_codes(k, rows, n, backward != 0);
    const bool dense = gated_dense(type, t, rows, n, backward != 0);
    plan[0] = dense ? 3 : c.sums.waves ? 1 : 2;
    plan[1] = dense ? sums_plan(block_terms(type), k, rows, n).splits : c.sums.splits;
    plan[2] = !backward ? 0 : dense ? grad_plan(block_terms(type), k, rows, n).splits : c.back.splits;
    return GPTQ_OK;
}

extern "C" size_t gptq_gated_workspace_size(int type, int64_t t, int64_t rows, int64_t n) { return gated_bytes(type, t, rows, n, false); }
extern "C" size_t gptq_gated_backward_workspace_size(int type, int64_t t, int64_t rows, int64_t n) {
    return gated_bytes(type, t, rows, n, true);
}

extern "C" int gptq_gated(const void* X, int64_t ldx, int type, int64_t t, int codec, const gptq_weights* gate,
                          const gptq_weights* up, int64_t rows, int64_t n, int act, void* Y, int64_t ldy, void* workspace,
                          size_t workspace_bytes, void* stream) {
    return gated_call(GatedCall{X, ldx, type, t, code_bits(codec), {gate, up}, rows, n, act, nullptr, 0, Y, ldy, workspace},
                      workspace_bytes, stream);
}

extern "C" int gptq_gated_backward(const void* dY, int64_t ldd, const void* X, int64_t ldx, int type, int64_t t, int codec,
                                   const gptq_weights* gate, const gptq_weights* up, int64_t rows, int64_t n, int act, void* dX,
                                   int64_t ldo, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dY && t) return GPTQ_EINVAL;
    return gated_call(GatedCall{X, ldx, type, t, code_bits(codec), {gate, up}, rows, n, act, dY, ldd, dX, ldo, workspace},
                      workspace_bytes, stream);
}
