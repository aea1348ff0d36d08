// backward.hip -- the gradient of a product's input, dX = dY W, from the sweeps' codes on gfx950.
//
// The sum runs over the rows of W, along which codes are not packed and every row has scales of its own.  So
// the scales join the gradients: of a group of 32 columns, dX = sum_r (dY[t][r] s[r]) (q[r][j] - z), with A = the
// scaled gradients of 16 tokens and 32 rows in two bf16 terms (16 bits), f32 in three, and B = the codes of 16
// columns as whole numbers (codes16.hpp); z and the operand's offset come out as A times a constant, for 16-bit results
// in a sum of their own, one for both tiles of a group, with no product waiting for another; the two meet every
// kJoinSteps steps.  (One term would do for bf16's own 8 bits, but puts a result as far off again as its last rounding
// does.)  In f32 B is the levels q - z themselves, exact in bf16 too: beside the offset's part its sums lost two bits to
// four (37 tokens of 2048 x 8192 in 2 bits 1.2e-6 off, a library's product of f32 0.8e-6).
//
// Two layouts: back_kernel on the codes; for many tokens in a 16-bit type W is turned and decoded to f16 and
// multiplied by dense16.hpp's tiled product.
#include "backward.hpp"

#include "../../include/gptq_check.h"
#include "check.hpp"
#include "dense16.hpp"

namespace gptq {

// Steps of a wave after which the offset's sums join the codes'.  Of gradients that do not cancel both grow with the rows
// on the way, 24 to 3 the result's root of them: joined at the end only, 17408 rows of one sign put an f16 result as far
// off as its rounding does (2.1e-4), 33000 twice that; every 512 rows of a wave leave 1e-5 at any number of rows.
constexpr int kJoinSteps = 16;

// Lane 2 J + (g >> 1) of each sixteen, in all of them: the scale of row 8 h + J and group g of a step.
template <int LANE>
__device__ __forceinline__ float broadcast16(float x) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x150 + LANE, 0xf, 0xf, false));
}

// The levels of the codes in bytes G of a and b as an operand's pair, exact.
template <int BITS, int G>
__device__ __forceinline__ uint32_t level_pair(uint32_t a, uint32_t b) {
    constexpr float z = BITS == 4 ? 8.0f : 1.5f;
    return pack_hi(__float_as_uint((float)(a >> (8 * G) & 255u) - z), __float_as_uint((float)(b >> (8 * G) & 255u) - z));
}

// A wave owns 128 columns (four groups) and 16 TT tokens; a step is 32 rows.  A lane (c, h) loads, of each of rows
// 8 h .. + 7, the word of eight codes of columns 8 c .. + 7, 64 bytes a row and quarter.  A matrix tile wants 16
// columns of one group, one a lane: the words' bytes are exchanged in two steps with lanes c ^ 8 and c ^ 7
// (each keeps the bytes whose number agrees with its own bit), which leaves byte g of a lane's word in group g, its
// two codes in columns 2 (4 d + 2 x + y) and the next, x and y the lane's bits 3 and 2, d its last two or, in groups
// of the other parity, 3 - d.  Rows two and two then make an operand's pairs as they are.
//
// The waves of a workgroup and the pieces of the grid's z take steps in turn; waves are joined in LDS.
// Bound by vector instructions around the products (the exchange, the scaled terms): 37 tokens of 2048 x 8192 in f32,
// 2 bits, 24 us and 4 to join, 333 of two 4096 x 2048 88; in 16 bits 100 to 130 TFLOP/s from 16 to 500 tokens.
template <int DD, int DT, int BITS, int TT, int NW>
__global__ __launch_bounds__(NW * 64, TT == 1 ? 4 : 2) void back_kernel(BackArgs a) {
    constexpr int TERMS = DT == GPTQ_F32 ? GPTQ_F32 : GPTQ_F16, NT = kTerms<TERMS>;
    __shared__ float red[NW / 2][TT * 32][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    // Workgroups go to the 8 XCDs in turn: each gets neighbouring columns, whose codes and scales share cache lines.
    const int g0 = ((blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3)) * 4, tok0 = blockIdx.y * 16 * TT;
    if (g0 >= a.G) return;
    const int there = min(4, a.G - g0);  // groups of these columns
    const int per = (a.rows + 31) / 32, all = per * a.mats;
    const int first = (int)((int64_t)all * blockIdx.z / gridDim.z) + wave, end = (int)((int64_t)all * (blockIdx.z + 1) / gridDim.z);
    // Words and scales of groups that are not there are those of ones that are.
    const int64_t bytes = (int64_t)a.G * (4 * BITS), word = (int64_t)g0 * (4 * BITS) + min(c, 4 * there - 1) * BITS;
    const int sg0 = g0 + min(2 * (c & 1), there - 1), sg1 = g0 + min(2 * (c & 1) + 1, there - 1);
    const uint32_t sel1 = c & 8 ? 0x03020706u : 0x05040100u, sel2 = c & 4 ? 0x03070105u : 0x06020400u;
    const u32v4 offset = BITS == 4 ? u32v4{kMinus24, kMinus24, kMinus24, kMinus24}
                                   : u32v4{0xC18CC18Cu, 0xC18CC18Cu, 0xC18CC18Cu, 0xC18CC18Cu};  // -17.5 = -(16 + 1.5)
    constexpr bool LEVELS = DT == GPTQ_F32;
    constexpr bool APART = !LEVELS && (DD != GPTQ_F32 || TT < 3);  // (else registers are short)
    f32v4 acc[TT][4][2], fix[APART ? TT : 1][4];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            acc[t][g][0] = acc[t][g][1] = f32v4{0.f, 0.f, 0.f, 0.f};
            fix[APART ? t : 0][g] = f32v4{0.f, 0.f, 0.f, 0.f};
        }

    struct Step {
        uint32_t w[8];
        float s[2];
        Raw<DD> x[TT];
        int r0;
    };
    auto load = [&](Step& k, int s) {
        const int m = s >= per ? 1 : 0;
        k.r0 = 32 * (s - m * per) + 8 * h;
        const uint8_t* codes = (m ? a.codes[1] : a.codes[0]) + word;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint8_t* p = codes + min(k.r0 + j, a.rows - 1) * bytes;
            k.w[j] = BITS == 4 ? *(const uint32_t*)p : (uint32_t)*(const uint16_t*)p;
        }
        const float* sp = (m ? a.scale[1] : a.scale[0]) + (int64_t)min(k.r0 + (c >> 1), a.rows - 1) * a.G;
        k.s[0] = sp[sg0];
        k.s[1] = sp[sg1];
#pragma unroll
        for (int t = 0; t < TT; ++t)
            k.x[t].load(a.D, (int64_t)min(tok0 + t * 16 + c, a.t - 1) * a.ldd + (int64_t)m * a.side + min(k.r0, (a.rows - 1) & ~7));
    };
    auto multiply = [&](Step& k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t x = k.w[j];
            if constexpr (BITS == 2) {  // a nibble a code
                x = (x | x << 8) & 0x00ff00ffu;
                x = (x | x << 4) & 0x0f0f0f0fu;
                x = (x | x << 2) & 0x33333333u;
            }
            const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xf, 0xf, false);  // lane c ^ 8
            x = __builtin_amdgcn_perm(y, x, sel1);
            const uint32_t z = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xf, 0xf, false);  // lane c ^ 7
            k.w[j] = __builtin_amdgcn_perm(z, x, sel2);
        }
        float d[TT][8];
#pragma unroll
        for (int t = 0; t < TT; ++t) k.x[t].floats(d[t]);
        if (__ballot(k.r0 + 8 > a.rows)) {  // rows that are not there
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int j = 0; j < 8; ++j) d[t][j] = k.r0 + j < a.rows ? d[t][j] : 0.0f;
        }
        auto group = [&](auto number) {
            constexpr int g = decltype(number)::value;
            u32v4 code[2];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                if constexpr (LEVELS) {
                    code[0][p] = level_pair<BITS, g>(k.w[2 * p] & 0x0f0f0f0fu, k.w[2 * p + 1] & 0x0f0f0f0fu);
                    code[1][p] = level_pair<BITS, g>(k.w[2 * p] >> 4 & 0x0f0f0f0fu, k.w[2 * p + 1] >> 4 & 0x0f0f0f0fu);
                    continue;
                }
                const uint32_t x = __builtin_amdgcn_perm(k.w[2 * p + 1], k.w[2 * p], 0x0c040c00u | g << 16 | g);
                code[0][p] = nibble_pair<0>(x);
                code[1][p] = nibble_pair<1>(x);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const float s = k.s[g & 1];
                float v[8] = {d[t][0] * broadcast16<(g >> 1)>(s),      d[t][1] * broadcast16<2 + (g >> 1)>(s),
                              d[t][2] * broadcast16<4 + (g >> 1)>(s),  d[t][3] * broadcast16<6 + (g >> 1)>(s),
                              d[t][4] * broadcast16<8 + (g >> 1)>(s),  d[t][5] * broadcast16<10 + (g >> 1)>(s),
                              d[t][6] * broadcast16<12 + (g >> 1)>(s), d[t][7] * broadcast16<14 + (g >> 1)>(s)};
                u32v4 terms[NT];
                weight_terms<TERMS>(v, terms);
                if constexpr (LEVELS) {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {  // a step's sum first, from its small terms up: fewer roundings at acc's size
                        f32v4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int e = NT - 1; e >= 0; --e) z = mfma16(terms[e], code[p], z);
                        acc[t][g][p] += z;
                    }
                } else if constexpr (APART) {
#pragma unroll
                    for (int e = 0; e < NT; ++e) {
                        acc[t][g][0] = mfma16(terms[e], code[0], acc[t][g][0]);
                        acc[t][g][1] = mfma16(terms[e], code[1], acc[t][g][1]);
                        fix[t][g] = mfma16(terms[e], offset, fix[t][g]);
                    }
                } else {
                    f32v4 start = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < NT; ++e) start = mfma16(terms[e], offset, start);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        f32v4 z = start;
#pragma unroll
                        for (int e = 0; e < NT; ++e) z = mfma16(terms[e], code[p], z);
                        acc[t][g][p] += z;
                    }
                }
                __builtin_amdgcn_sched_barrier(0);  // one token tile's operands at a time
            }
        };
        group(std::integral_constant<int, 0>{});
        group(std::integral_constant<int, 1>{});
        group(std::integral_constant<int, 2>{});
        group(std::integral_constant<int, 3>{});
    };
    auto join = [&]() {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                acc[t][g][0] += fix[t][g];
                acc[t][g][1] += fix[t][g];
                fix[t][g] = f32v4{0.f, 0.f, 0.f, 0.f};
            }
    };
    Step now, next;
    if (first < end) load(now, first);
    int turn = 0;
    for (int s = first; s < end; s += NW) {
        load(next, min(s + NW, end - 1));
        multiply(now);
        now = next;
        if constexpr (APART)
            if (++turn % kJoinSteps == 0) join();
    }
    if constexpr (APART) join();
    // Waves two and two: the upper half hands its sums to the lower, until one is left.
#pragma unroll
    for (int n = NW / 2; n >= 1; n /= 2) {
        if (wave >= n && wave < 2 * n) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int u = 0; u < 32; ++u) red[wave - n][t * 32 + u][lane] = acc[t][u >> 3][u >> 2 & 1][u & 3];
        }
        __syncthreads();
        if (wave < n) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int u = 0; u < 32; ++u) acc[t][u >> 3][u >> 2 & 1][u & 3] += red[wave][t * 32 + u][lane];
        }
        __syncthreads();
    }
    if (wave) return;
    const int x = c >> 3, y = c >> 2 & 1, d = c & 3;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        if (g >= there) break;
        const int col = 32 * (g0 + g) + 2 * (4 * ((g & 1) == y ? d : 3 - d) + 2 * x + y);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tok = tok0 + t * 16 + 4 * h + r;
                if (tok >= a.t) continue;
                const float z0 = acc[t][g][0][r], z1 = acc[t][g][1][r];
                if (a.part) {
                    *(f32v2*)(a.part + ((int64_t)blockIdx.z * a.t + tok) * a.n + col) = f32v2{z0, z1};
                } else {
                    store_one<DT>(a.Y, (int64_t)tok * a.ldy + col, z0);
                    store_one<DT>(a.Y, (int64_t)tok * a.ldy + col + 1, z1);
                }
            }
    }
}

// The sums of the pieces, in their order: four columns a thread.
template <int DT>
__global__ __launch_bounds__(256) void back_join_kernel(BackArgs a, int splits) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, n = (int64_t)a.t * a.n;
    if (i >= n) return;
    f32v4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int s = 0; s < splits; ++s) z += *(const f32v4*)(a.part + s * n + i);
    const int64_t tok = i / a.n, col = i - tok * a.n;
#pragma unroll
    for (int k = 0; k < 4; ++k) store_one<DT>(a.Y, tok * a.ldy + col + k, z[k]);
}

// dY with rows of whole 16 bytes, its own columns only: zeros behind them.
template <int DT>
__global__ __launch_bounds__(256) void pad_kernel(const void* X, int64_t ld, int n, void* P, int64_t ldp) {
    const int64_t tok = blockIdx.x;
    for (int i = threadIdx.x; i < ldp; i += 256) store_one<DT>(P, tok * ldp + i, i < n ? load_one<DT>(X, tok * ld + i) : 0.0f);
}

typedef void (*BackKernel)(BackArgs);
template <int DD, int DT, int BITS>
static BackKernel back_pick(const BackPlan& p) {
    return p.tt == 1 ? back_kernel<DD, DT, BITS, 1, 4> : p.tt == 2 ? back_kernel<DD, DT, BITS, 2, 4> : back_kernel<DD, DT, BITS, 3, 4>;
}
template <int DD, int DT>
static BackKernel back_pick(const BackPlan& p, int bits) {
    return bits == 4 ? back_pick<DD, DT, 4>(p) : back_pick<DD, DT, 2>(p);
}

// Tiles of 16 tokens a wave, and pieces of the rows: what a call takes is taken to be the rounds of workgroups that the
// CUs hold (four, with more tiles two) times a wave's steps and two more that a piece costs beside them; a wave keeps
// two or three.  Measured (us, f32 unless said otherwise):
//   tiles   one, two, three a wave, 2048 x 8192: 16 tokens 13.8, 16.7, 20; 37 25, 26, 24; 128 50, 41, 50; 333 112, 98, 79
//   waves   one token of 5120 x 17408, bf16: eight of a workgroup 33, sixteen 45, four 28.5
BackPlan back_plan(int64_t t, int64_t rows, int mats, int64_t n) {
    BackPlan p{t <= 16 ? 1 : t <= 128 ? 2 : 3, 4, 1};
    if (p.tt == 3 && (t + 47) / 48 * 3 > (t + 31) / 32 * 2 + (t + 31) / 32 / 4) p.tt = 2;  // too many left empty
    const int64_t steps = (rows + 31) / 32 * mats, wg = (n + 127) / 128 * ((t + 16 * p.tt - 1) / (16 * p.tt));
    const int64_t hold = (p.tt == 1 ? 4 : 2) * kCUs, most = steps / ((p.tt == 1 ? 2 : 3) * p.waves);
    double best = 0.0;
    for (int64_t s = 1; s == 1 || (s <= most && (s - 1) * wg < 2 * hold); ++s) {
        const double cost = (double)((s * wg + hold - 1) / hold) * ((double)((steps + s * p.waves - 1) / (s * p.waves)) + 2.0) + (s > 1 ? 1.0 + 0.05 * (double)s : 0.0);
        if (s == 1 || cost < best) {
            best = cost;
            p.splits = (int)s;
        }
    }
    return p;
}

int back_run(BackArgs a, const BackPlan& p, int dd, int dt, int bits, hipStream_t st) {
    const BackKernel k = dt == GPTQ_F32    ? back_pick<GPTQ_F32, GPTQ_F32>(p, bits)
                         : dt == GPTQ_BF16 ? (dd == GPTQ_F32 ? back_pick<GPTQ_F32, GPTQ_BF16>(p, bits) : back_pick<GPTQ_BF16, GPTQ_BF16>(p, bits))
                                           : (dd == GPTQ_F32 ? back_pick<GPTQ_F32, GPTQ_F16>(p, bits) : back_pick<GPTQ_F16, GPTQ_F16>(p, bits));
    void (*const join)(BackArgs, int) = dt == GPTQ_F32 ? back_join_kernel<GPTQ_F32> : dt == GPTQ_BF16 ? back_join_kernel<GPTQ_BF16> : back_join_kernel<GPTQ_F16>;
    const int64_t des = dtype_size(dd), es = dtype_size(dt), cb = (int64_t)a.G * 4 * bits;
    if (p.splits < 2) a.part = nullptr;
    const dim3 grid((unsigned)round_up((a.G + 3) / 4, 8), (unsigned)((a.t + 16 * p.tt - 1) / (16 * p.tt)), (unsigned)p.splits);
    const int64_t wide = (a.mats - 1) * (int64_t)a.side + a.rows;
    ProfScope ps(FAM_LINEAR, st, 2.0 * (double)a.t * a.rows * a.n * a.mats, (double)a.mats * a.rows * (cb + 4 * a.G));
    GPTQ_LAUNCH(st, "linear_back", (k<<<grid, p.waves * 64, 0, st>>>(a)), rd(a.D, a.ldd, a.t, wide, (int)des),
                rd(a.codes[0], cb, a.rows, cb, 1), rd(a.scale[0], a.G, a.rows, a.G),
                rd(a.codes[a.mats - 1], cb, a.rows, cb, 1), rd(a.scale[a.mats - 1], a.G, a.rows, a.G),
                wr(a.part ? (const void*)a.part : a.Y, a.part ? a.n : a.ldy, a.part ? (int64_t)a.t * p.splits : a.t, a.n, a.part ? 4 : (int)es));
    if (a.part)
        GPTQ_LAUNCH(st, "linear_back_join", (join<<<(unsigned)(((int64_t)a.t * a.n / 4 + 255) / 256), 256, 0, st>>>(a, p.splits)),
                    rd(a.part, a.n, (int64_t)a.t * p.splits, a.n), wr(a.Y, a.ldy, a.t, a.n, (int)es));
    return GPTQ_OK;
}

// Many tokens in a 16-bit type run on decoded weights, where there is enough to multiply for four launches.  Measured (us,
// codes / decoded, bf16; tokens of rows x n):
//   100 of 5120 x 17408 132 / 136, 200 of them 213 / 135; 150 of 4096 x 4096 (2.5e9 products) 39 / 46, 200 (3.4e9)
//   50 / 44; 512 of 4096 x 1024 (2.1e9) 37 / 40, 1000 of 2048 x 2048 (4.2e9) 59 / 41; 2500 of 2500 x 512 (3.2e9) 93 / 58.
// f16 takes the same within a tenth.
static bool back_dense(int type, int64_t t, int64_t rows, int64_t n) {
    return (type == GPTQ_BF16 || type == GPTQ_F16) && t > 128 && t * rows * n > 2800000000 && rows <= (1 << 21);
}
struct BackSpace {
    int64_t side, slice;  // columns of D; tokens at once
    size_t token, D, W, part, bytes;
};
static BackSpace back_space(int64_t t, int64_t rows, int64_t n) {
    BackSpace s;
    s.side = round_up(rows, kTileK);
    s.slice = t < kTokens16 ? t : kTokens16;
    s.token = align256(4 * (size_t)rows);  // the rows' powers before it
    s.D = s.token + align256(4 * (size_t)s.slice);
    s.W = s.D + align256(2 * (size_t)s.slice * (size_t)s.side);
    s.part = s.W + align256(2 * (size_t)round_up(n, kTileR) * (size_t)s.side);
    s.bytes = s.part;
    for (int64_t k : {s.slice, t % s.slice}) {
        if (!k) continue;
        const DensePlan p = dense16_plan(k, n, s.side);
        const size_t b = s.part + sizeof(float) * (size_t)((p.tiles - p.whole) * p.splits) * (kTileT * kTileR);
        if (b > s.bytes) s.bytes = b;
    }
    return s;
}
static int64_t pad_ld(int64_t rows) { return round_up(rows, 8); }
// The codes' product: kTokens16 tokens at a time, their gradients with padded rows, then the pieces' sums.
static size_t pad_bytes(int dtype, int64_t t, int64_t rows) { return align256((size_t)dtype_size(dtype) * (size_t)t * (size_t)pad_ld(rows)); }
static size_t codes_bytes(int dtype, int64_t t, int64_t rows, int64_t n) {
    return pad_bytes(dtype, t, rows) + back_part_bytes(back_plan(t, rows, 1, n), t, n);
}

template <int DT>
static int back_dense_run(const void* dY, int64_t ldd, const BackArgs& b, int bits, void* workspace, hipStream_t st) {
    const int64_t t = b.t, rows = b.rows, n = b.n, cb = (int64_t)b.G * 4 * bits;
    const BackSpace s = back_space(t, rows, n);
    char* ws = (char*)workspace;
    float* power = (float*)ws;
    float* token = (float*)(ws + s.token);
    uint16_t* D = (uint16_t*)(ws + s.D);
    uint16_t* W = (uint16_t*)(ws + s.W);
    const Turn turn{{b.codes[0], b.codes[0]}, {b.scale[0], b.scale[0]}, power, false, (int)rows, (int)n, (int)s.side, (int)s.side, W};
    ProfScope ps(FAM_LINEAR, st, 2.0 * (double)t * rows * n, 0.0);
    GPTQ_LAUNCH(st, "row_power", (row_power_kernel<<<(unsigned)rows, 256, 0, st>>>(b.scale[0], b.G, power)),
                rd(b.scale[0], b.G, rows, b.G), wr(power, rows, 1, rows));
    const dim3 grid((unsigned)((n + 255) / 256), (unsigned)(s.side / 64), 1);
    GPTQ_LAUNCH(st, "linear_turn", (bits == 4 ? turn_kernel<4><<<grid, 256, 0, st>>>(turn) : turn_kernel<2><<<grid, 256, 0, st>>>(turn)),
                rd(b.codes[0], cb, rows, cb, 1), rd(b.scale[0], b.G, rows, b.G), rd(power, rows, 1, rows), wr(W, s.side, n, s.side, 2));
    for (int64_t t0 = 0; t0 < t; t0 += s.slice) {
        const int64_t k = t - t0 < s.slice ? t - t0 : s.slice;
        const DensePlan p = dense16_plan(k, n, s.side);
        const int64_t cut = (p.tiles - p.whole) * p.splits, sums = cut * kTileT * kTileR;
        const Halve hv{(const char*)dY + t0 * ldd * 2, ldd, (int)rows, power, D, (int)s.side, token, nullptr, nullptr};
        GPTQ_LAUNCH(st, "linear_halve", (halve_kernel<DT><<<(unsigned)k, 256, 0, st>>>(hv)), rd(hv.X, ldd, k, rows, 2),
                    rd(power, rows, 1, rows), wr(D, s.side, k, s.side, 2), wr(token, k, 1, k));
        Dense16 d{};
        d.X = D;
        d.ldx = (int)s.side;
        d.t = (int)k;
        d.W = W;
        d.ldw = (int)s.side;
        d.token = token;
        d.rows = (int)n;
        d.Y = (char*)b.Y + t0 * b.ldy * 2;
        d.ldy = b.ldy;
        d.tiles_r = (int)p.tiles_r;
        d.tiles = (int)p.tiles;
        d.whole = (int)p.whole;
        d.splits = (int)p.splits;
        d.part = (float*)(ws + s.part);
        GPTQ_LAUNCH(st, "linear_dense16", (dense16_kernel<DT, DENSE_PLAIN><<<(unsigned)(p.whole + cut), kDenseWaves * 64, 0, st>>>(d)),
                    rd(D, s.side, k, s.side, 2), rd(W, s.side, round_up(n, kTileR), s.side, 2), rd(token, k, 1, k),
                    wr(d.Y, d.ldy, k, n, 2), wr(d.part, sums, cut ? 1 : 0, sums));
        if (cut)
            GPTQ_LAUNCH(st, "linear_dense16_join",
                        (dense16_join_kernel<DT, DENSE_PLAIN><<<dim3(kTileT * kTileR / 1024, (unsigned)(p.tiles - p.whole)), 256, 0, st>>>(d)),
                        rd(d.part, sums, 1, sums), rd(token, k, 1, k), wr(d.Y, d.ldy, k, n, 2));
    }
    return GPTQ_OK;
}

static bool back_sizes_ok(int dtype, int64_t t, int64_t rows, int64_t n) {
    return dtype_size(dtype) && t >= 0 && t <= (1 << 24) && rows >= 1 && rows <= (1 << 23) && t * rows <= ((int64_t)1 << 38) &&
           n >= 32 && n <= (1 << 20) && n % 32 == 0 && t * n <= ((int64_t)1 << 38);
}

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_check_backward_plan(int type, int64_t t, int64_t rows, int64_t n, int64_t* plan) {
    if (!plan || !back_sizes_ok(type & ~GPTQ_EXACT_WEIGHTS, t, rows, n) || t == 0) return GPTQ_EINVAL;
    const bool dense = back_dense(type, t, rows, n);
    const int64_t k = t < kTokens16 ? t : kTokens16;
    const BackPlan c = back_plan(k, rows, 1, n);
    plan[0] = dense ? 3 : 1;
    plan[1] = dense ? dense16_plan(k, n, round_up(rows, kTileK)).splits : c.splits;
    plan[2] = dense ? 0 : c.tt;
    return GPTQ_OK;
}

extern "C" size_t gptq_linear_backward_workspace_size(int type, int64_t t, int64_t rows, int64_t n) {
    const int dtype = type & ~GPTQ_EXACT_WEIGHTS;
    if (!back_sizes_ok(dtype, t, rows, n) || t == 0) return 0;
    if (back_dense(type, t, rows, n)) return back_space(t, rows, n).bytes;
    size_t most = 0;
    for (int64_t k : {t < kTokens16 ? t : kTokens16, t % kTokens16})
        if (k && codes_bytes(dtype, k, rows, n) > most) most = codes_bytes(dtype, k, rows, n);
    return most;
}

extern "C" int gptq_linear_backward(const void* dY, int64_t ldd, int type, int64_t t, int codec, const uint8_t* codes,
                                    const float* scale, int64_t rows, int64_t n, void* dX, int64_t ldx, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    const int dtype = type & ~GPTQ_EXACT_WEIGHTS;
    if (!back_sizes_ok(dtype, t, rows, n)) return GPTQ_EINVAL;
    if (codec != GPTQ_CODEC_Q4TP && codec != GPTQ_CODEC_Q2TP) return GPTQ_EINVAL;
    if (t == 0) return GPTQ_OK;
    const int es = dtype_size(dtype), bits = codec == GPTQ_CODEC_Q4TP ? 4 : 2;
    if (!dY || !codes || !scale || !dX || ldd < rows || ldx < n || ldd > ((int64_t)1 << 36) || ldx > ((int64_t)1 << 36)) return GPTQ_EINVAL;
    if (!al16(codes) || ((uintptr_t)scale & 3u) || ((uintptr_t)dY | (uintptr_t)dX) % (unsigned)es) return GPTQ_EINVAL;
    const size_t need = gptq_linear_backward_workspace_size(type, t, rows, n);
    if (!workspace || workspace_bytes < need) return GPTQ_EWORKSPACE;
    if ((uintptr_t)workspace & 255u) return GPTQ_EINVAL;
    const int64_t G = n / 32, cb = G * 4 * bits;
    const RowSet x{dX, ldx * es, t, n * es}, w{workspace, (int64_t)need, 1, (int64_t)need};
    const RowSet in[] = {RowSet{dY, ldd * es, t, rows * es}, RowSet{codes, rows * cb, 1, rows * cb}, RowSet{scale, rows * G * 4, 1, rows * G * 4}};
    if (rows_meet(x, w)) return GPTQ_EINVAL;
    for (const RowSet& i : in)
        if (rows_meet(x, i) || rows_meet(w, i)) return GPTQ_EINVAL;
    CheckScope check;
    check_buffer(workspace, workspace_bytes, "workspace");
    check_buffer(dY, (size_t)es * (size_t)((t - 1) * ldd + rows), "dY");
    check_buffer(codes, (size_t)(rows * cb), "codes");
    check_buffer(scale, sizeof(float) * (size_t)(rows * G), "scale");
    check_buffer(dX, (size_t)es * (size_t)((t - 1) * ldx + n), "dX");
    hipStream_t st = (hipStream_t)stream;
    BackArgs a{dY, ldd, 0, 1, (int)rows, (int)G, (int)n, {codes, codes}, {scale, scale}, (int)t, dX, ldx, nullptr};
    int rc;
    if (back_dense(type, t, rows, n)) {
        rc = dtype == GPTQ_BF16 ? back_dense_run<GPTQ_BF16>(dY, ldd, a, bits, workspace, st)
                                : back_dense_run<GPTQ_F16>(dY, ldd, a, bits, workspace, st);
    } else {
        const bool padded = rows % 8 || !al16(dY) || ldd % (16 / es);
        const int64_t ldp = pad_ld(rows);
        void (*const pad)(const void*, int64_t, int, void*, int64_t) =
            dtype == GPTQ_F32 ? pad_kernel<GPTQ_F32> : dtype == GPTQ_BF16 ? pad_kernel<GPTQ_BF16> : pad_kernel<GPTQ_F16>;
        rc = GPTQ_OK;
        for (int64_t t0 = 0; t0 < t && rc == GPTQ_OK; t0 += kTokens16) {
            const int64_t k = t - t0 < kTokens16 ? t - t0 : kTokens16;
            BackArgs b = a;
            b.t = (int)k;
            b.D = (const char*)dY + t0 * ldd * es;
            b.Y = (char*)dX + t0 * ldx * es;
            if (padded) {
                GPTQ_LAUNCH(st, "linear_pad", (pad<<<(unsigned)k, 256, 0, st>>>(b.D, ldd, (int)rows, workspace, ldp)), rd(b.D, ldd, k, rows, es),
                            wr(workspace, ldp, k, ldp, es));
                b.D = workspace;
                b.ldd = ldp;
            }
            b.part = (float*)((char*)workspace + pad_bytes(dtype, k, rows));
            rc = back_run(b, back_plan(k, rows, 1, n), dtype, dtype, bits, st);
        }
    }
    if (rc != GPTQ_OK) return rc;
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}
