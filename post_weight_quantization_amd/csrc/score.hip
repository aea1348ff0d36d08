// score.hip -- the attention that cached tokens have received, on gfx950.
//
//   score[t] = old[t] + sum over the call's rows and a kv head's query heads of e^(scale q k_t - lse),
// lse the row's own (gptq_cache_attention's): the softmax weights of the whole call, added up by token.
//
// Tokens own the work: a wave holds the keys of 16 TT tokens of one kv head and walks over the query rows that see
// them, 16 at a time.  Scores come with queries in D's rows and tokens in its columns, so a lane adds up four
// queries of one token of each tile, and the quarters of the wave are added at the end.  Nothing is joined
// through memory, and results do not depend on timing.  A lane adds four weights in f32 and, with many rows, their sums in
// f64 (two instructions a turn), so that a token's sum keeps f32's bits over any number of rows; in f32 throughout 32768
// query rows were 2.1e-7 off, half of it by log2 e rounded to f32.
//
// Few rows (decoding): the codes are multiplied as whole numbers and scaled afterwards, as in
// attention_rows_kernel.  Many rows, or f32: keys are decoded once to bf16, where c s is exact, and stay in
// registers; bound by vector instructions, the exponentials above all, one a score and four times as long as another.
#include <math.h>

#include "attention.hpp"

namespace gptq {

struct ScoreArgs {
    AttnArgs a;        // lse is read here
    const float* old;  // [pages, heads, page]
    float* out;        // the same places; may be old itself
    int tiles;         // workgroups along a sequence; each takes every tiles-th piece of it
};

constexpr int kScoreSlots = 4;   // waves of a workgroup side by side on a sequence's tokens: few rows
constexpr int kTileSlots = 2, kTileShares = 4;  // .. and those that share the rows of the same tokens: many rows
constexpr int kTileRows = 16 * kTileShares;      // query rows in LDS at a time
template <int G>
constexpr int kScoreTiles = G == 8 ? 2 : 4;  // 16-token tiles of a wave: decoded keys in 64 registers (dim 64: 32)

template <int G>
constexpr int kRowsTiles = 8 / G;   // .. of a wave with few rows, twice on their way

// lse log2 e, log2 e to 48 bits: rounded to 24 every weight of a row were off the same way.
__device__ __forceinline__ float log2_of(float lse) { return fmaf(lse, 1.4426950408889634f, lse * 1.9259629911e-8f); }

// Query rows (counted row * group + head) that see a token of [tok0, tok1) at all: a range that holds them.
__host__ __device__ __forceinline__ void score_rows(int tok0, int tok1, int pos0, int R, int group, int window, int sinks,
                                                    int& x0, int& x1) {
    const int64_t first = (int64_t)tok0 - pos0;  // the first row at or behind tok0
    int64_t last = R;
    if (window && tok0 >= sinks) {
        const int64_t past = (int64_t)tok1 - 1 + window - pos0;  // the first row whose window has left tok1 - 1
        if (past < last) last = past;
    }
    const int64_t a = first > 0 ? first : 0, b = last > a ? last : a;
    x0 = a < R ? (int)(a * group) : R * group;
    x1 = b < R ? (int)(b * group) : R * group;
}

// Few rows: a wave takes pieces of 16 TT tokens, kScoreSlots times `tiles` pieces apart, the next one's codes on their
// way while it multiplies the present one's.
template <int DT, int G>
__global__ __launch_bounds__(kScoreSlots * 64, G == 8 ? 2 : G == 4 && DT == GPTQ_F16 ? 3 : 4) void score_rows_kernel(ScoreArgs s) {
    constexpr int NT = kTerms<DT>, TT = kRowsTiles<G>, TOK = 16 * TT;
    const AttnArgs& a = s.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int head = blockIdx.x % a.c.heads, first = blockIdx.x / a.c.heads;
    const int b = blockIdx.y + blockIdx.z * kGridTiles;
    if (b >= a.q.seqs) return;
    int r0, r1;
    seq_rows(a.q, b, r0, r1);
    const int R = __builtin_amdgcn_readfirstlane(r1 - r0);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    const int64_t held = (int64_t)a.q.width * a.c.page;
    const int len = __builtin_amdgcn_readfirstlane(max(a.q.len[b], 0)), pos0 = len - R, end = (int)min((int64_t)len, held);
    const int32_t* table = a.q.table + (int64_t)b * a.q.width;
    const u32v4 minus24 = {kMinus24, kMinus24, kMinus24, kMinus24};
    const int pieces = (int)(((int64_t)end + TOK - 1) / TOK), step = s.tiles * kScoreSlots;
    int piece = first * kScoreSlots + wave;
    if (piece >= pieces) return;

    struct Keys {
        uint32_t w[TT][G], s[TT][G / 2];
        int64_t place;  // of this lane's token tok0 + 16 h + c
        float old;
        bool writes;
    };
    auto fetch = [&](Keys& k, int v) {
        const int tok0 = v * TOK;
        bool there = false;
#pragma unroll
        for (int u = 0; u < TT; ++u) {
            bool is;
            const int64_t at = find_page(a, table, head, tok0 + 16 * u, is);
            load_key_words<G>(a.c.k + (at + c) * (16 * G) + h * (4 * G), k.w[u]);
            const uint32_t* sp = (const uint32_t*)(a.c.ks + (at + c) * G);
#pragma unroll
            for (int i = 0; i < G / 2; ++i) k.s[u][i] = sp[i];
            if (h == u) {
                k.place = at + c;
                there = is;
            }
        }
        const int tok = tok0 + 16 * h + c;
        k.writes = there && h < TT && tok < end;
        k.old = k.writes && tok < pos0 ? s.old[k.place] : 0.0f;
    };
    // Sixteen queries from x on: terms, what the codes' offset adds, and of this lane's four their bases and positions.
    const int X = R * a.group;
    u32v4 q[G][NT];
    f32v4 start[G];
    float base2[4];
    int qpos[4], q0 = 0, q1 = 0;
    auto queries = [&](int x) {
        const int xq = min(x + c, X - 1), qi = xq / a.group, qh = head * a.group + (xq - qi * a.group);
        const int64_t row = r0 + qi;
        const float lse = a.lse[row * a.qheads + qh];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            load_terms<DT, false>(a.Q, row * a.ldq + (int64_t)qh * a.ldqh + 32 * i + 8 * h, q[i]);
#pragma unroll
            for (int k = 0; k < NT; ++k) q[i][k] ^= a.flip;
            start[i] = f32v4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < NT; ++k) start[i] = mfma16(q[i][k], minus24, start[i]);
        }
        // A row that sees nothing has lse = -inf and pays nothing; nor does one behind the last.
        float less = log2_of(lse);
        if (lse == -INFINITY || x + c >= X) less = INFINITY;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            base2[r] = -__shfl(less, 20 * h + r);
            qpos[r] = pos0 + __shfl(qi, 20 * h + r);
        }
        q0 = __builtin_amdgcn_readlane(qi, 0);
        q1 = __builtin_amdgcn_readlane(qi, 15);
    };
    Keys now, next;
    fetch(now, piece);
    if (X > 0) queries(0);
    for (; piece < pieces; piece += step) {
        fetch(next, min(piece + step, pieces - 1));
        const int tok0 = piece * TOK;
        float sum[TT];
#pragma unroll
        for (int u = 0; u < TT; ++u) sum[u] = 0.0f;
        int x0, x1;
        score_rows(tok0, tok0 + TOK, pos0, R, a.group, a.window, a.sinks, x0, x1);
        for (int x = x0 & ~15; x < x1; x += 16) {
            if (X > 16) queries(x);
            f32v4 d[TT];
#pragma unroll
            for (int u = 0; u < TT; ++u) d[u] = f32v4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < G; ++i) {
#pragma unroll
                for (int u = 0; u < TT; ++u) {
                    uint32_t w = now.w[u][i];
                    asm volatile("" : "+v"(w));  // unpacked here: ahead of the loop it takes 64 registers
                    const u32v4 codes = unpack_nibbles(w);
                    const uint32_t y = now.s[u][i >> 1];
                    const float scale = __uint_as_float((i & 1) ? y & 0xffff0000u : y << 16);
                    f32v4 z = start[i];
#pragma unroll
                    for (int k = 0; k < NT; ++k) z = mfma16(q[i][k], codes, z);
#pragma unroll
                    for (int r = 0; r < 4; ++r) d[u][r] = fmaf(scale, z[r], d[u][r]);
                }
                __builtin_amdgcn_sched_barrier(0);  // one group's operands at a time
            }
            const bool inner = tok0 + TOK - 1 <= pos0 + q0 && (window_low(pos0 + q1, a.window) < tok0 || tok0 + TOK <= a.sinks);
#pragma unroll
            for (int u = 0; u < TT; ++u) {
                float part = 0.0f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(d[u][r], a.scale2, base2[r]));
                    const bool seen = inner || key_seen(tok0 + 16 * u + c, qpos[r], window_low(qpos[r], a.window), a.sinks);
                    part += seen ? p : 0.0f;
                }
                sum[u] += part;
            }
        }
        float paid = 0.0f;
#pragma unroll
        for (int u = 0; u < TT; ++u) {
            const float all = quad_sum(sum[u]);
            if (h == u) paid = all;
        }
        if (now.writes) s.out[now.place] = now.old + paid;
        now = next;
    }
}

// Many rows, or f32.  kTileSlots waves side by side hold the decoded keys of 16 TT tokens each; kTileShares of them the
// same ones, for every kTileShares-th 16 of the rows.  Rows come to LDS, straight from memory, one turn ahead:
// loaded by each wave for itself they took 131 us (2 x up to 1000 rows of 16 heads over 8192 tokens), most of it
// waiting, and 93 so, 430 TFLOP/s.  Eight waves, two a SIMD: with six the barrier waited for the SIMDs with two (115).  A row's
// 16-byte pieces lie in LDS in an order that its low bits permute, so that operand reads touch all banks.
template <int DT, int G>
__global__ __launch_bounds__(kTileSlots * kTileShares * 64, G == 2 ? 4 : 2) void score_tile_kernel(ScoreArgs s) {
    constexpr int NT = kTerms<DT>, TT = kScoreTiles<G>, TOK = 16 * TT, WAVES = kTileSlots * kTileShares;
    constexpr int ES = DT == GPTQ_F32 ? 4 : 2, P = 32 * G * ES / 16;  // 16-byte pieces of a row
    constexpr int LOADS = kTileRows * P / (64 * WAVES);               // of a wave and turn, 64 / P rows each
    static_assert(LOADS * 64 * WAVES == kTileRows * P && 64 % P == 0, "whole loads of whole rows");
    // Arrays of their own for the turn that is read and the one that is loaded: of one array's halves the compiler
    // waits for the loads of the one before it reads the other.
    __shared__ u32v4 rows0[kTileRows * P], rows1[kTileRows * P];
    __shared__ __attribute__((aligned(16))) float less0[kTileRows], less1[kTileRows];
    __shared__ __attribute__((aligned(16))) int qpos0[kTileRows], qpos1[kTileRows];
    __shared__ float red[kTileShares - 1][kTileSlots][TT][64];
    const AttnArgs& a = s.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = wave % kTileSlots, share = wave / kTileSlots;
    const int c = lane & 15, h = lane >> 4;
    const int head = blockIdx.x / s.tiles, first = blockIdx.x - head * s.tiles;
    const int b = blockIdx.y + blockIdx.z * kGridTiles;
    if (b >= a.q.seqs) return;
    int r0, r1;
    seq_rows(a.q, b, r0, r1);
    const int R = __builtin_amdgcn_readfirstlane(r1 - r0);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    const int64_t held = (int64_t)a.q.width * a.c.page;
    const int len = __builtin_amdgcn_readfirstlane(max(a.q.len[b], 0)), pos0 = len - R, end = (int)min((int64_t)len, held);
    const int32_t* table = a.q.table + (int64_t)b * a.q.width;
    constexpr int WIDE = kTileSlots * TOK;
    for (int64_t at = (int64_t)first * WIDE; at < end; at += (int64_t)s.tiles * WIDE) {
        const int tok0 = (int)min(at + slot * TOK, (int64_t)(end - 1) / TOK * TOK);  // behind the end the last again, not written
        int x0, x1;
        score_rows((int)at, (int)at + WIDE, pos0, R, a.group, a.window, a.sinks, x0, x1);
        // Where this lane loads from in the next turn: row `mine[k]` of it and its offset, moved on by a turn's rows and,
        // where the head passes the group's last, to the next row's first.  The last row stands for those behind it.
        const int step_q = kTileRows / a.group, step_r = kTileRows - step_q * a.group;
        const int last_q = (x1 - 1) / a.group, last_r = x1 - 1 - last_q * a.group;
        const int64_t go = step_q * a.ldq + step_r * a.ldqh, wrap = a.ldq - a.group * a.ldqh;
        const int64_t last = (r0 + last_q) * a.ldq + (int64_t)(head * a.group + last_r) * a.ldqh;
        int64_t from[LOADS];
        int rem[LOADS], lse_q = 0, lse_r = 0;
        auto begin = [&](int x, int row, int& q, int& r) {
            const int xq = min(x + row, x1 - 1);
            q = xq / a.group;
            r = xq - q * a.group;
        };
        auto row_of = [&](int k) { return (wave * LOADS + k) * 64 / P + lane / P; };
        auto fetch = [&](int x, u32v4* rows) {
#pragma unroll
            for (int k = 0; k < LOADS; ++k) {
                const int row = row_of(k), piece = (lane % P) ^ (row & (P - 1) & 15);
                const int64_t off = x + row < x1 ? from[k] : last;
                __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) const void*)((const char*)a.Q + off * ES + 16 * piece),
                                                 (__attribute__((address_space(3))) void*)(rows + (wave * LOADS + k) * 64), 16, 0, 0);
                from[k] += go;
                rem[k] += step_r;
                if (rem[k] >= a.group) {
                    rem[k] -= a.group;
                    from[k] += wrap;
                }
            }
        };
        // A wave's loads to LDS are done before it comes to the barrier behind which the others read them.
        auto rows_there = [&]() {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
        };
        // Of row threadIdx.x of a turn: what its weights' exponents begin with, and its position.
        float lse = 0.0f;
        int at_pos = 0;
        bool pays = false;
        auto fetch_lse = [&](int x) {
            if (threadIdx.x >= kTileRows) return;
            pays = x + (int)threadIdx.x < x1;
            const int q = pays ? lse_q : last_q, r = pays ? lse_r : last_r;
            lse = a.lse[(int64_t)(r0 + q) * a.qheads + head * a.group + r];
            at_pos = pos0 + q;
            lse_q += step_q;
            lse_r += step_r;
            if (lse_r >= a.group) {
                lse_r -= a.group;
                ++lse_q;
            }
        };
        auto keep_lse = [&](float* less, int* qpos) {
            if (threadIdx.x >= kTileRows) return;
            // A row that sees nothing has lse = -inf and pays nothing; nor does one behind the last.
            less[threadIdx.x] = pays && lse != -INFINITY ? -log2_of(lse) : -INFINITY;
            qpos[threadIdx.x] = at_pos;
        };
        if (x0 < x1) {
#pragma unroll
            for (int k = 0; k < LOADS; ++k) {
                int q;
                begin(x0, row_of(k), q, rem[k]);
                from[k] = (r0 + q) * a.ldq + (int64_t)(head * a.group + rem[k]) * a.ldqh;
            }
            begin(x0, threadIdx.x, lse_q, lse_r);
            fetch(x0, rows0);
            fetch_lse(x0);
        }
        u32v4 key[TT][G];
        int64_t place = 0;
        bool there = false;
#pragma unroll
        for (int u = 0; u < TT; ++u) {
            bool is;
            const int64_t row = find_page(a, table, head, tok0 + 16 * u, is);
            uint32_t w[G];
            load_key_words<G>(a.c.k + (row + c) * (16 * G) + h * (4 * G), w);
            const uint32_t* sp = (const uint32_t*)(a.c.ks + (row + c) * G);
            if (h == u) {
                place = row + c;
                there = is;
            }
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const uint32_t y = sp[i >> 1];
                const float z = __uint_as_float((i & 1) ? y & 0xffff0000u : y << 16), z8 = -8.0f * z;
                const uint32_t even = nibble_bytes(w[i], false), odd = nibble_bytes(w[i], true);
                key[u][i] = u32v4{decode_pair<0, 2>(even, z, z8, z, z8), decode_pair<0, 2>(odd, z, z8, z, z8),
                                  decode_pair<1, 3>(even, z, z8, z, z8), decode_pair<1, 3>(odd, z, z8, z, z8)} ^ a.flip;
            }
        }
        // Token tok0 + 16 h + c is this lane's to write (TT tiles; the first TT quarters).
        const int tok = tok0 + 16 * h + c;
        const bool writes = there && h < TT && tok < end && at + slot * TOK < end && share == 0;
        const float old = writes && tok < pos0 ? s.old[place] : 0.0f;
        keep_lse(less0, qpos0);
        rows_there();

        double sum[TT];
#pragma unroll
        for (int u = 0; u < TT; ++u) sum[u] = 0.0;
        auto turn = [&](int x, const u32v4* rows, const float* less, const int* qpos, u32v4* rows_n, float* less_n, int* qpos_n) {
            const bool more = x + kTileRows < x1;
            if (more) {
                fetch(x + kTileRows, rows_n);
                fetch_lse(x + kTileRows);
            }
            __builtin_amdgcn_sched_barrier(0);
            f32v4 d[TT];
#pragma unroll
            for (int u = 0; u < TT; ++u) d[u] = f32v4{0.f, 0.f, 0.f, 0.f};
            const u32v4* mine = rows + (share * 16 + c) * P;
#pragma unroll
            for (int i = 0; i < G; ++i) {
                u32v4 raw[ES / 2], q[NT];
#pragma unroll
                for (int k = 0; k < ES / 2; ++k) raw[k] = mine[((ES / 2) * (4 * i + h) + k) ^ (c & (P - 1))];
                raw_terms<DT, false>(raw, q);
#pragma unroll
                for (int k = 0; k < NT; ++k)
#pragma unroll
                    for (int u = 0; u < TT; ++u) d[u] = mfma16(q[k], key[u][i], d[u]);
            }
            // D's rows are queries 4 h + r of the sixteen.
            const f32v4 base2 = *(const f32v4*)(less + share * 16 + 4 * h);
            const int q0 = __builtin_amdgcn_readfirstlane(qpos[share * 16]), q1 = __builtin_amdgcn_readfirstlane(qpos[share * 16 + 15]);
            if (tok0 + TOK - 1 <= q0 && (window_low(q1, a.window) < tok0 || tok0 + TOK <= a.sinks)) {  // all of them see all
#pragma unroll
                for (int u = 0; u < TT; ++u) {
                    float p[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) p[r] = __builtin_amdgcn_exp2f(fmaf(d[u][r], a.scale2, base2[r]));
                    sum[u] += (p[0] + p[1]) + (p[2] + p[3]);
                }
            } else {
                float part[TT][2];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int pos = qpos[share * 16 + 4 * h + r], low = window_low(pos, a.window);
#pragma unroll
                    for (int u = 0; u < TT; ++u) {
                        const float p = __builtin_amdgcn_exp2f(fmaf(d[u][r], a.scale2, base2[r]));
                        const float x = key_seen(tok0 + 16 * u + c, pos, low, a.sinks) ? p : 0.0f;
                        part[u][r >> 1] = r & 1 ? part[u][r >> 1] + x : x;
                    }
                }
#pragma unroll
                for (int u = 0; u < TT; ++u) sum[u] += part[u][0] + part[u][1];
            }
            if (more) keep_lse(less_n, qpos_n);
            rows_there();
        };
        for (int x = x0; x < x1; x += 2 * kTileRows) {
            turn(x, rows0, less0, qpos0, rows1, less1, qpos1);
            if (x + kTileRows < x1) turn(x + kTileRows, rows1, less1, qpos1, rows0, less0, qpos0);
        }
        float all[TT];
#pragma unroll
        for (int u = 0; u < TT; ++u) all[u] = (float)sum[u];
        if (share > 0)
#pragma unroll
            for (int u = 0; u < TT; ++u) red[share - 1][slot][u][lane] = all[u];
        __syncthreads();
        float paid = 0.0f;
#pragma unroll
        for (int u = 0; u < TT; ++u) {
            if (share == 0)
#pragma unroll
                for (int k = 0; k + 1 < kTileShares; ++k) all[u] += red[k][slot][u][lane];
            const float z = quad_sum(all[u]);
            if (h == u) paid = z;
        }
        if (writes) s.out[place] = old + paid;
        __syncthreads();
    }
}

typedef void (*ScoreKernel)(ScoreArgs);
template <int DT>
static ScoreKernel score_pick(int dim, bool few) {
    if constexpr (DT != GPTQ_F32)
        if (few) return dim == 64 ? score_rows_kernel<DT, 2> : dim == 128 ? score_rows_kernel<DT, 4> : score_rows_kernel<DT, 8>;
    return dim == 64 ? score_tile_kernel<DT, 2> : dim == 128 ? score_tile_kernel<DT, 4> : score_tile_kernel<DT, 8>;
}

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_cache_score(const gptq_cache* cache, const gptq_batch* batch, const void* Q, int64_t ldq, int64_t ldqh,
                                int32_t q_heads, int dtype, float scale, int32_t window, int32_t sinks, const float* lse,
                                const float* score, float* out, void* stream) {
    const int es = dtype_size(dtype);
    if (!es || !cache_ok(cache) || !batch_ok(batch) || !table_ok(cache, batch) || !qheads_ok(cache, q_heads)) return GPTQ_EINVAL;
    if (!isfinite(scale) || window < 0 || sinks < 0) return GPTQ_EINVAL;
    if (!score || !out || (((uintptr_t)lse | (uintptr_t)score | (uintptr_t)out) & 3u)) return GPTQ_EINVAL;
    if (batch->rows && (!Q || !lse || !heads_ok(Q, batch->rows, ldq, ldqh, q_heads, cache->dim, es))) return GPTQ_EINVAL;
    const int group = q_heads / cache->heads;
    if (batch->rows * group > ((int64_t)1 << 27)) return GPTQ_EINVAL;
    const int64_t tokens = cache->pages * cache->page * cache->heads, items = batch->rows * q_heads;
    // Old scores are read by the workgroup that writes them: out is score, or shares nothing with it.
    const RowSet o{out, 4 * tokens, 1, 4 * tokens};
    if (out != score && rows_meet(o, RowSet{score, 4 * tokens, 1, 4 * tokens})) return GPTQ_EINVAL;
    const int64_t seq_bytes = 4 * (int64_t)batch->seqs;
    if (rows_meet(o, RowSet{batch->table, seq_bytes * batch->width, 1, seq_bytes * batch->width}) ||
        rows_meet(o, RowSet{batch->len, seq_bytes, 1, seq_bytes}) ||
        rows_meet(o, RowSet{batch->start, seq_bytes + 4, batch->start ? 1 : 0, seq_bytes + 4}))
        return GPTQ_EINVAL;
    if (meets_cache(o, cache) || rows_meet(o, RowSet{lse, 4 * items, items ? 1 : 0, 4 * items}) ||
        rows_meet(o, heads_rows(Q, batch->rows, ldq, ldqh, q_heads, cache->dim, es)))
        return GPTQ_EINVAL;
    CheckScope check;
    check_cache(cache, batch);
    if (batch->rows) {
        check_buffer(Q, heads_bytes(batch->rows, ldq, ldqh, q_heads, cache->dim, es), "Q");
        check_buffer(lse, sizeof(float) * (size_t)items, "lse");
    }
    check_buffer(score, sizeof(float) * (size_t)tokens, "score");
    if (out != score) check_buffer(out, sizeof(float) * (size_t)tokens, "out");
    hipStream_t st = (hipStream_t)stream;
    ScoreArgs s{AttnArgs{cache_view(cache), batch_view(batch), Q, ldq, ldqh, q_heads, group,
                         (float)fmin(fmax(fabs((double)scale) * 1.4426950408889634, 0x1p-100), 0x1p127),
                         scale < 0.0f ? 0x80008000u : 0u, window, sinks, nullptr, 0, 0, const_cast<float*>(lse), nullptr, 1,
                         page_div(cache->page).m, page_div(cache->page).shift},
                score, out, 1};
    // By the rows a sequence on average, which is what the host knows.  Measured (us, score_rows_kernel / score_tile_kernel; 8
    // heads of 128 in bf16 over 4096 tokens, 8 query heads each): 64 single rows 49 / 381, 64 sequences of 4 rows 106 / 396, 8 of
    // 8 34 / 57; one of 4 over 2000 tokens 12 / 12, of 16 15 / 12.  A batch of both kinds can lose: 63 single rows and
    // a chunk of 190 867 / 430; 512 and one of 4000 over 512 tokens, a query head each, 11400 / 800.
    const bool few = dtype != GPTQ_F32 && batch->rows * group <= 32 * (int64_t)batch->seqs;
    const int64_t piece = few ? kScoreSlots * 16 * (256 / cache->dim) : kTileSlots * 16 * (cache->dim == 256 ? 2 : 4);
    int64_t tiles = ((int64_t)batch->width * cache->page + piece - 1) / piece;
    // Workgroups past a grid's size, or many rounds of them: each takes several pieces of its sequence.
    int64_t most = ((int64_t)1 << 20) / ((int64_t)cache->heads * (batch->seqs < 16 ? batch->seqs : 16)) + 1;
    if (few) {
        const int64_t hold = 8 * kCUs, lists = (int64_t)cache->heads * batch->seqs;
        most = lists < hold ? (hold + lists - 1) / lists : 1;
    }
    if (tiles > most) tiles = most;
    s.tiles = (int)tiles;
    const ScoreKernel k = dtype == GPTQ_F32    ? score_pick<GPTQ_F32>(cache->dim, false)
                          : dtype == GPTQ_BF16 ? score_pick<GPTQ_BF16>(cache->dim, few)
                                               : score_pick<GPTQ_F16>(cache->dim, few);
    const int64_t qw = (q_heads - 1) * ldqh + cache->dim, seqs = batch->seqs;
    const Span none = rd(score, tokens, 0, tokens);
    {
        ProfScope ps(FAM_ATTENTION, st, 0.0, 0.0);
        GPTQ_LAUNCH(st, "cache_score",
                    (k<<<dim3((unsigned)(cache->heads * tiles), (unsigned)(seqs < kGridTiles ? seqs : kGridTiles),
                              (unsigned)((seqs + kGridTiles - 1) / kGridTiles)), (few ? kScoreSlots : kTileSlots * kTileShares) * 64, 0, st>>>(s)),
                    batch->rows ? rd(Q, ldq, batch->rows, qw, es) : none, batch->rows ? rd(lse, items, 1, items) : none,
                    batch_span(batch, 0), batch_span(batch, 1), batch_span(batch, 2), plane(cache->k, cache, cache->dim / 2, false),
                    plane(cache->k_scale, cache, cache->dim / 16, false), rd(score, tokens, 1, tokens), wr(out, tokens, 1, tokens));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}
