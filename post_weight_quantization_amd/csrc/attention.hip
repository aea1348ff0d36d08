// attention.hip -- attention over the 4-bit cache on gfx950.
//
//   o = softmax(scale q K^T) V,  K = c s (key codes c, one s per token and 32 channels), V alike.
//
// The codes are multiplied as whole numbers (codes16.hpp): for a group i of 32 channels one
// 16x16x32 MFMA gives sum_d (c_d + 24) q_d for 16 tokens and 16 query rows, started from -24 sum_d q_d,
// and the score adds s_i times that, in f32.  For the values the scale is the token's, so it joins
// the softmax weight: with p' = p s_i rounded to bf16 (one, two or three terms for bf16, f16, f32),
// o_d = sum_t p'_t (c_td + 24) - 24 sum_t p'_t; the second sum is one more MFMA of the same p'
// against a constant operand, so that the rounding of p' meets only c, not the offset.
//
// Scores are made transposed, tokens in D's rows and queries in its columns.  A lane then holds
// eight scores of one query over two 16-token tiles, which is the layout the second product wants
// its weights in (the order of tokens inside a product is free as long as V's operand has the same),
// and the running maximum and sum of a query are scalars of its four lanes.
//
// attention_rows_kernel: a workgroup owns 16 query rows (the query heads of one kv head, times the
// rows of one sequence) and a piece of the sequence; its four waves take 32 tokens at a time and
// are joined in LDS.  Where rows are few the sequence is cut into `splits` pieces, whose partial sums
// attention_join_kernel adds, in a fixed order.
#include <math.h>

#include "../../include/gptq_check.h"
#include "cache.hpp"

namespace gptq {

struct AttnArgs {
    CacheView c;
    Batch q;
    const void* Q;
    int64_t ldq, ldqh;
    int qheads, group;
    float scale2;  // scale times log2 e: the softmax runs on powers of two
    int window, sinks;
    void* O;
    int64_t ldo, ldoh;
    float* lse;
    float* part;     // [splits][rows][qheads][dim], then [splits][rows][qheads] of (maximum, sum)
    int splits;
};

constexpr int kAttnWaves = 4;
constexpr int kBlock = 32;      // tokens a wave takes at a time
constexpr int kRowsTile = 16;   // query rows of a workgroup
constexpr int kMinBlocks = 8;   // 32-token blocks of a piece at least

// Where a tile of query rows stands: its sequence, rows and the blocks of 32 tokens it looks at.
struct Tile {
    int b, r0, R;      // sequence, its first row, its rows
    int x0;            // first of the tile's query rows, counted row * group + head of the group
    int pos0;          // position of row r0 (may be negative)
    int lo_blk;        // first block of the window
    int sink_blks;     // blocks of sinks before it
    int blks;          // all blocks
    int end;           // tokens at `end` and past it are seen by no row
    int64_t all_lo;    // every row sees the tokens from all_lo on (and below `sinks`) ..
    int all_hi;        // .. that are before all_hi
};

// L tokens cached, `held` of them can have pages.  All arithmetic that could pass 31 bits is 64.
__host__ __device__ __forceinline__ void tile_blocks(int L, int64_t held, int group, int window, int sinks,
                                                     int rows_tile, Tile& t) {
    L = L > 0 ? L : 0;
    t.pos0 = L - t.R;
    const int q0 = t.x0 / group, last = (t.x0 + rows_tile - 1) / group, q1 = last < t.R - 1 ? last : t.R - 1;
    const int64_t end = (int64_t)t.pos0 + q1 + 1 < held ? (int64_t)t.pos0 + q1 + 1 : held;
    t.end = end > 0 ? (int)end : 0;
    const int64_t low = window ? (int64_t)t.pos0 + q0 - window + 1 : 0;
    t.lo_blk = low > 0 ? (int)(low / kBlock) : 0;
    const int end_blk = (int)(((int64_t)t.end + kBlock - 1) / kBlock);
    const int before = t.lo_blk < end_blk ? t.lo_blk : end_blk;
    const int sink = window ? (int)(((int64_t)sinks + kBlock - 1) / kBlock) : 0;
    t.sink_blks = sink < before ? sink : before;
    t.blks = t.sink_blks + (end_blk > t.lo_blk ? end_blk - t.lo_blk : 0);
    t.all_lo = window ? (int64_t)t.pos0 + q1 - window + 1 : 0;
    t.all_hi = t.pos0 + q0 + 1 < t.end ? t.pos0 + q0 + 1 : t.end;
}
// Block v of the tile's, as a block of the sequence.
__host__ __device__ __forceinline__ int tile_block(const Tile& t, int v) {
    return v < t.sink_blks ? v : t.lo_blk + (v - t.sink_blks);
}
// Does every row of the tile see all of a block's tokens?
__host__ __device__ __forceinline__ bool block_inner(const Tile& t, int tok0, int tokens, int sinks) {
    return tok0 + tokens <= t.all_hi && (tok0 >= t.all_lo || tok0 + tokens <= sinks);
}
// A row at qpos sees the tokens up to qpos that are past `window_low` of it, or sinks.
__host__ __device__ __forceinline__ int window_low(int qpos, int window) {
    return window && qpos >= window ? qpos - window : -1;
}
__host__ __device__ __forceinline__ bool key_seen(int tok, int qpos, int low, int sinks) {
    return (tok <= qpos) & ((tok > low) | (tok < sinks));
}
// Blocks of one piece: the sequence's blocks over the splits, whole turns of the waves.
__host__ __device__ __forceinline__ int piece_blocks(int blks, int splits) {
    int per = (blks + splits - 1) / splits;
    if (per < kMinBlocks) per = kMinBlocks;
    return (per + kAttnWaves - 1) / kAttnWaves * kAttnWaves;
}
__device__ __forceinline__ void tile_of_call(const AttnArgs& a, int rows_tile, Tile& t) {
    tile_blocks(a.q.len[t.b], (int64_t)a.q.width * a.c.page, a.group, a.window, a.sinks, rows_tile, t);
}

// The tile of a workgroup: sequences in order, ceil(R group / rows_tile) tiles each.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int rows_tile, int x, Tile& t) {
    if (!a.q.start) {
        const int per = (a.group + rows_tile - 1) / rows_tile;
        t.b = x / per;
        t.r0 = t.b;
        t.R = 1;
        t.x0 = (x - t.b * per) * rows_tile;
        return true;
    }
    const int lane = threadIdx.x & 63;
    for (int b0 = 0; b0 < a.q.seqs; b0 += 64) {
        int r0 = 0, r1 = 0;
        if (b0 + lane < a.q.seqs) seq_rows(a.q, b0 + lane, r0, r1);
        const int n = (int)(((int64_t)(r1 - r0) * a.group + rows_tile - 1) / rows_tile);
        int sum = n;
#pragma unroll
        for (int k = 1; k < 64; k *= 2) {
            const int y = __shfl_up(sum, k);
            if (lane >= k) sum += y;
        }
        const unsigned long long past = __ballot(sum > x);
        if (past) {
            const int l = __builtin_ctzll(past);
            t.b = b0 + l;
            t.r0 = __shfl(r0, l);
            t.R = __shfl(r1, l) - t.r0;
            t.x0 = (x - (__shfl(sum, l) - __shfl(n, l))) * rows_tile;
            return true;
        }
        x -= __shfl(sum, 63);
    }
    return false;
}

// Word i of a key's or value's G bytes a lane: loads of G bytes (values) or 4 G bytes (keys).
template <int G>
__device__ __forceinline__ void load_key_words(const uint8_t* p, uint32_t (&w)[G]) {
    if constexpr (G == 2) {
        const u32v2 v = *(const u32v2*)p;
        w[0] = v[0];
        w[1] = v[1];
    } else {
#pragma unroll
        for (int k = 0; k < G / 4; ++k) {
            const u32v4 v = ((const u32v4*)p)[k];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * k + j] = v[j];
        }
    }
}
// The G scales of four tokens in a row as floats: s[r][i].
template <int G>
__device__ __forceinline__ void load_scales(const uint16_t* p, float (&s)[4][G]) {
    uint32_t w[2 * G];
#pragma unroll
    for (int k = 0; k < G / 2; ++k) {
        const u32v4 v = ((const u32v4*)p)[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * k + j] = v[j];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const uint32_t x = w[(r * G + i) >> 1];
            s[r][i] = __uint_as_float((i & 1) ? x & 0xffff0000u : x << 16);
        }
}
// G bytes of a value row as G / 2 halves of 16 bits: half j in the low bits of w[j].
template <int G>
__device__ __forceinline__ void load_value_words(const uint8_t* p, uint32_t (&w)[(G + 3) / 4]) {
    if constexpr (G == 2) w[0] = *(const uint16_t*)p;
    if constexpr (G == 4) w[0] = *(const uint32_t*)p;
    if constexpr (G == 8) {
        const u32v2 v = *(const u32v2*)p;
        w[0] = v[0];
        w[1] = v[1];
    }
}

// Eight weights as kTerms operands, the last rounded to nearest even.
template <int DT>
__device__ __forceinline__ void weight_terms(float (&v)[8], u32v4 (&t)[kTerms<DT>]) {
#pragma unroll
    for (int s = 0; s + 1 < kTerms<DT>; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t b0 = __float_as_uint(v[2 * k]), b1 = __float_as_uint(v[2 * k + 1]);
            t[s][k] = pack_hi(b0, b1);
            v[2 * k] -= __uint_as_float(b0 & 0xffff0000u);
            v[2 * k + 1] -= __uint_as_float(b1 & 0xffff0000u);
        }
#pragma unroll
    for (int k = 0; k < 4; ++k) t[kTerms<DT> - 1][k] = round_bf16x2(v[2 * k], v[2 * k + 1]);
}

template <int DT, int G>
__global__ __launch_bounds__(kAttnWaves * 64) void attention_rows_kernel(AttnArgs a) {
    constexpr int NT = kTerms<DT>;
    constexpr int D = 32 * G;
    __shared__ float joined[kAttnWaves][2 * G][64][4];
    __shared__ float stat[kAttnWaves][2][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, h = lane >> 4;
    const int head = blockIdx.y, split = blockIdx.z;
    Tile t;
    if (!find_tile(a, kRowsTile, blockIdx.x, t)) return;
    tile_of_call(a, kRowsTile, t);
    const int per = piece_blocks(t.blks, a.splits);
    const int v0 = split * per, v1 = min(t.blks, v0 + per);
    if (v0 >= v1 && split != 0) return;
    const bool whole = t.blks <= per;

    // This lane's query row.
    const int xq = min(t.x0 + c, t.R * a.group - 1);
    const int qi = xq / a.group, qh = head * a.group + (xq - qi * a.group);
    const int qpos = t.pos0 + qi, low = window_low(qpos, a.window);
    u32v4 q[G][NT];
    f32v4 start[G];
    const u32v4 minus24 = {kMinus24, kMinus24, kMinus24, kMinus24};
#pragma unroll
    for (int i = 0; i < G; ++i) {
        load_terms<DT, false>(a.Q, (int64_t)(t.r0 + qi) * a.ldq + (int64_t)qh * a.ldqh + 32 * i + 8 * h, q[i]);
        start[i] = f32v4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NT; ++k) start[i] = mfma16(minus24, q[i][k], start[i]);
    }
    f32v4 o[G][2], fix[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
        o[i][0] = f32v4{0.f, 0.f, 0.f, 0.f};
        o[i][1] = o[i][0];
        fix[i] = o[i][0];
    }
    float m = -INFINITY, l = 0.0f;
    const int32_t* table = a.q.table + (int64_t)t.b * a.q.width;
    for (int v = v0 + wave; v < v1; v += kAttnWaves) {
        const int tok0 = tile_block(t, v) * kBlock;
        int64_t place[2];
        bool there[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int tok = tok0 + 16 * u;
            int page = -1;
            const int at = tok / a.c.page;
            if (at < a.q.width) page = table[at];
            there[u] = (unsigned)page < (unsigned)a.c.pages;
            place[u] = ((int64_t)(there[u] ? page : 0) * a.c.heads + head) * a.c.page + (tok - at * a.c.page);
        }
        uint32_t kw[2][G], vw[2][4][(G + 3) / 4];
        float ks[2][4][G], vs[2][4][G];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            load_key_words<G>(a.c.k + (place[u] + c) * (16 * G) + h * (4 * G), kw[u]);
            load_scales<G>(a.c.ks + (place[u] + 4 * h) * G, ks[u]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                load_value_words<G>(a.c.v + (place[u] + 4 * h + r) * (16 * G) + c * G, vw[u][r]);
            load_scales<G>(a.c.vs + (place[u] + 4 * h) * G, vs[u]);
        }
        float p[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f32v4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const u32v4 kk = unpack_nibbles(kw[u][i]);
                f32v4 d = start[i];
#pragma unroll
                for (int k = 0; k < NT; ++k) d = mfma16(kk, q[i][k], d);
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] = fmaf(ks[u][r][i], d[r], s[r]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) p[4 * u + r] = s[r] * a.scale2;
        }
        // Blocks at an edge of what the rows see (or with an absent page): score by score.  Selects, not
        // branches around the assignments: under branches the compiler keeps the unmasked scores.
        const bool inner = there[0] && there[1] && block_inner(t, tok0, kBlock, a.sinks);
        unsigned hidden = 0u;
        if (!inner) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int tok = tok0 + 16 * (j >> 2) + 4 * h + (j & 3);
                const bool seen = there[j >> 2] & key_seen(tok, qpos, low, a.sinks);
                hidden |= seen ? 0u : 1u << j;
                p[j] = seen ? p[j] : -INFINITY;
            }
        }
        float top = p[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = fmaxf(top, p[j]);
        top = fmaxf(m, quad_max(top));
        if (__ballot(top > m)) {
            const float less = m == top ? 1.0f : exp2f(m - top);
            m = top;
            l *= less;
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    o[i][0][r] *= less;
                    o[i][1][r] *= less;
                    fix[i][r] *= less;
                }
        }
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] = exp2f(p[j] - base);
            l += p[j];
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            // Weights times the group's scales; a hidden token's scale may be anything.
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = p[j] * vs[j >> 2][j & 3][i];
            if (!inner) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = (hidden >> j & 1u) ? 0.0f : w[j];
            }
            u32v4 pt[NT];
            weight_terms<DT>(w, pt);
#pragma unroll
            for (int k = 0; k < NT; ++k) fix[i] = mfma16(minus24, pt[k], fix[i]);
            // Codes of group i, channels m and 16 + m: nibbles 2 (i % 2) and the next of half i / 2.
            u32v4 c0, c1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int u = k >> 1, r = 2 * (k & 1), word = i >> 2;
                const uint32_t x = (i >> 1 & 1) ? pack_hi(vw[u][r][word], vw[u][r + 1][word])
                                                : pack_lo(vw[u][r][word], vw[u][r + 1][word]);
                c0[k] = (i & 1) ? nibble_pair<2>(x) : nibble_pair<0>(x);
                c1[k] = (i & 1) ? nibble_pair<3>(x) : nibble_pair<1>(x);
            }
#pragma unroll
            for (int k = 0; k < NT; ++k) {
                o[i][0] = mfma16(c0, pt[k], o[i][0]);
                o[i][1] = mfma16(c1, pt[k], o[i][1]);
            }
        }
    }

    // Join the waves: a common maximum per query, sums in wave order.
    l = quad_sum(l);
    if (h == 0) {
        stat[wave][0][c] = m;
        stat[wave][1][c] = l;
    }
    __syncthreads();
    float M = -INFINITY, Lsum = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) M = fmaxf(M, stat[w][0][c]);
    const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) Lsum += stat[w][1][c] * exp2f(stat[w][0][c] - base);
    const float mine = exp2f(m - base);
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) joined[wave][2 * i + n][lane][r] = (o[i][n][r] + fix[i][r]) * mine;
    __syncthreads();
    const bool real = t.x0 + c < t.R * a.group;
    const int64_t row = t.r0 + qi, item = row * a.qheads + qh;
    const float inv = Lsum == 0.0f ? 0.0f : 1.0f / Lsum;
    for (int u = wave; u < 2 * G; u += kAttnWaves) {
        float y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float x = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttnWaves; ++w) x += joined[w][u][lane][r];
            y[r] = whole ? x * inv : x;
        }
        const int d = 16 * u + 4 * h;  // channels 32 i + 16 n + 4 h ..
        if (!real) continue;
        if (whole)
            store_four<DT>(a.O, row * a.ldo + (int64_t)qh * a.ldoh + d, y);
        else
            *(f32v4*)(a.part + ((int64_t)split * a.q.rows * a.qheads + item) * D + d) = f32v4{y[0], y[1], y[2], y[3]};
    }
    if (real && wave == 0 && h == 0) {
        if (!whole) {
            float* ml = a.part + (int64_t)a.splits * a.q.rows * a.qheads * D +
                        2 * ((int64_t)split * a.q.rows * a.qheads + item);
            ml[0] = M;
            ml[1] = Lsum;
        } else if (a.lse) {
            a.lse[item] = Lsum == 0.0f ? -INFINITY : (M + log2f(Lsum)) * 0.69314718055994531f;
        }
    }
}

// One wave per row and query head: the pieces' sums over a common maximum, in order.
template <int DT, int G>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
    constexpr int D = 32 * G, E = D / 64;
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (item >= a.q.rows * a.qheads) return;
    const int row = (int)(item / a.qheads), qh = (int)(item - (int64_t)row * a.qheads);
    Tile t;
    t.b = seq_of_row(a.q, row);
    if (t.b < 0) return;
    int r1;
    seq_rows(a.q, t.b, t.r0, r1);
    t.R = r1 - t.r0;
    t.x0 = ((row - t.r0) * a.group + qh % a.group) / kRowsTile * kRowsTile;
    tile_of_call(a, kRowsTile, t);
    const int per = piece_blocks(t.blks, a.splits);
    if (t.blks <= per) return;  // written whole
    const int n = (t.blks + per - 1) / per;
    const int64_t step = a.q.rows * a.qheads;
    const float* ml = a.part + (int64_t)a.splits * step * D + 2 * item;
    float M = -INFINITY;
    for (int s = 0; s < n; ++s) M = fmaxf(M, ml[2 * s * step]);
    const float base = M == -INFINITY ? 0.0f : M;
    float L = 0.0f, y[E] = {};
    for (int s = 0; s < n; ++s) {
        const float w = exp2f(ml[2 * s * step] - base);
        L += ml[2 * s * step + 1] * w;
        const float* p = a.part + (s * step + item) * D + E * lane;
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = fmaf(p[e], w, y[e]);
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int e = 0; e < E; ++e)
        store_one<DT>(a.O, row * a.ldo + (int64_t)qh * a.ldoh + E * lane + e, y[e] * inv);
    if (a.lse && lane == 0) a.lse[item] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

typedef void (*AttnKernel)(AttnArgs);
template <int DT>
static void attn_kernels(int dim, AttnKernel& rows, AttnKernel& join) {
    rows = dim == 64    ? attention_rows_kernel<DT, 2>
           : dim == 128 ? attention_rows_kernel<DT, 4>
                        : attention_rows_kernel<DT, 8>;
    join = dim == 64    ? attention_join_kernel<DT, 2>
           : dim == 128 ? attention_join_kernel<DT, 4>
                        : attention_join_kernel<DT, 8>;
}

// Tiles of rows_tile query rows of one kv head, at most: each sequence may end in a part of one.
static int64_t tiles_at_most(const gptq_batch* b, int group, int rows_tile) {
    if (!b->start) return (int64_t)b->seqs * ((group + rows_tile - 1) / rows_tile);
    const int64_t most = (b->rows * group + rows_tile - 1) / rows_tile + b->seqs;
    return most < b->rows * group ? most : b->rows * group;
}
// Pieces a sequence is cut into, so that about four workgroups a CU are there to hide latency,
// while a piece keeps kMinBlocks blocks of the longest sequence the table can hold.
static int attn_splits(const gptq_cache* c, const gptq_batch* b, int group) {
    const int64_t wg = tiles_at_most(b, group, kRowsTile) * c->heads;
    const int64_t blks = ((int64_t)b->width * c->page + kBlock - 1) / kBlock;
    int64_t s = wg > 0 ? (1024 + wg - 1) / wg : 1;
    const int64_t most = (blks + kMinBlocks - 1) / kMinBlocks;
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}
static size_t attn_part_bytes(const gptq_cache* c, const gptq_batch* b, int qheads, int splits) {
    return splits <= 1 ? 0 : align256(sizeof(float) * (size_t)splits * (size_t)b->rows * (size_t)qheads * (size_t)(c->dim + 2));
}
static bool qheads_ok(const gptq_cache* c, int qheads) {
    return qheads >= c->heads && qheads % c->heads == 0 && qheads / c->heads <= 64;
}

}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_cache_attention_workspace_size(const gptq_cache* cache, const gptq_batch* batch,
                                                      int32_t q_heads) {
    if (!cache || !batch_sizes_ok(batch) || cache->heads < 1 || cache->page < 16 || !qheads_ok(cache, q_heads)) return 0;
    return attn_part_bytes(cache, batch, q_heads, attn_splits(cache, batch, q_heads / cache->heads));
}

extern "C" int gptq_cache_attention(const gptq_cache* cache, const gptq_batch* batch, const void* Q, int64_t ldq,
                                    int64_t ldqh, int32_t q_heads, int dtype, float scale, int32_t window,
                                    int32_t sinks, void* O, int64_t ldo, int64_t ldoh, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    const int es = dtype_size(dtype);
    if (!es || !cache_ok(cache) || !batch_ok(batch) || !qheads_ok(cache, q_heads)) return GPTQ_EINVAL;
    if (!isfinite(scale) || window < 0 || sinks < 0) return GPTQ_EINVAL;
    if (batch->rows == 0) return GPTQ_OK;
    if (!Q || !O || !heads_ok(Q, batch->rows, ldq, ldqh, q_heads, cache->dim, es) ||
        !heads_ok(O, batch->rows, ldo, ldoh, q_heads, cache->dim, es) || ((uintptr_t)lse & 3u))
        return GPTQ_EINVAL;
    const int group = q_heads / cache->heads;
    if (batch->rows * group > ((int64_t)1 << 27)) return GPTQ_EINVAL;
    const int splits = attn_splits(cache, batch, group);
    const size_t need = attn_part_bytes(cache, batch, q_heads, splits);
    if (need) {
        if (!workspace || workspace_bytes < need) return GPTQ_EWORKSPACE;
        if (!al16(workspace)) return GPTQ_EINVAL;
    }
    CheckScope check;
    check_cache(cache, batch);
    check_buffer(Q, heads_bytes(batch->rows, ldq, ldqh, q_heads, cache->dim, es), "Q");
    check_buffer(O, heads_bytes(batch->rows, ldo, ldoh, q_heads, cache->dim, es), "O");
    if (lse) check_buffer(lse, sizeof(float) * (size_t)(batch->rows * q_heads), "lse");
    if (need) check_buffer(workspace, workspace_bytes, "workspace");
    hipStream_t st = (hipStream_t)stream;
    const AttnArgs a{cache_view(cache), batch_view(batch), Q, ldq, ldqh, q_heads, group,
                     (float)((double)scale * 1.4426950408889634), window, sinks, O, ldo, ldoh, lse, (float*)workspace,
                     splits};
    AttnKernel rows, join;
    if (dtype == GPTQ_F32)
        attn_kernels<GPTQ_F32>(cache->dim, rows, join);
    else if (dtype == GPTQ_BF16)
        attn_kernels<GPTQ_BF16>(cache->dim, rows, join);
    else
        attn_kernels<GPTQ_F16>(cache->dim, rows, join);
    const int64_t tiles = tiles_at_most(batch, group, kRowsTile);
    const int64_t items = batch->rows * q_heads;
    const int64_t qw = (q_heads - 1) * ldqh + cache->dim, ow = (q_heads - 1) * ldoh + cache->dim;
    const int64_t pf = (int64_t)(need / 4);
    {
        ProfScope ps(FAM_ATTENTION, st, 0.0, 0.0);
        GPTQ_LAUNCH(st, "attention_rows",
                    (rows<<<dim3((unsigned)tiles, (unsigned)cache->heads, (unsigned)splits), kAttnWaves * 64, 0, st>>>(a)),
                    rd(Q, ldq, batch->rows, qw, es), batch_span(batch, 0), batch_span(batch, 1), batch_span(batch, 2),
                    plane(cache->k, cache, cache->dim / 2, false), plane(cache->v, cache, cache->dim / 2, false),
                    plane(cache->k_scale, cache, cache->dim / 16, false),
                    plane(cache->v_scale, cache, cache->dim / 16, false), wr(O, ldo, batch->rows, ow, es),
                    wr(lse ? (const void*)lse : O, items, lse ? 1 : 0, items),
                    wr(need ? (const void*)workspace : O, pf, need ? 1 : 0, pf));
        if (splits > 1)
            GPTQ_LAUNCH(st, "attention_join", (join<<<(unsigned)((items + 3) / 4), 256, 0, st>>>(a)),
                        batch_span(batch, 1), batch_span(batch, 2), rd(workspace, pf, 1, pf),
                        wr(O, ldo, batch->rows, ow, es), wr(lse ? (const void*)lse : O, items, lse ? 1 : 0, items));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}

extern "C" int64_t gptq_check_cache_row(int64_t pages, int32_t page, int32_t heads, int32_t width,
                                        const int32_t* table, int32_t seq, int64_t pos, int32_t head) {
    CacheView c{};
    c.pages = (int)pages;
    c.page = page;
    c.heads = heads;
    Batch q{};
    q.table = table;
    q.width = width;
    return cache_row(c, q, seq, pos, head);
}

// Every key that a row of the sequence sees has to be in exactly one block of the row's tile, and
// every key of an inner block has to be seen by all of the tile's rows.
extern "C" int gptq_check_attention_blocks(int32_t len, int32_t rows, int32_t group, int64_t held, int32_t window,
                                           int32_t sinks, int32_t splits) {
    if (rows < 1 || group < 1 || held < 0 || window < 0 || sinks < 0 || splits < 1) return GPTQ_EINVAL;
    for (int x0 = 0; x0 < rows * group; x0 += kRowsTile) {
        Tile t{};
        t.R = rows;
        t.x0 = x0;
        tile_blocks(len, held, group, window, sinks, kRowsTile, t);
        const int per = piece_blocks(t.blks, splits);
        if ((int64_t)per * splits < t.blks || per % kAttnWaves) return GPTQ_ECHECK;
        for (int x = x0; x < x0 + kRowsTile && x < rows * group; ++x) {
            const int qpos = t.pos0 + x / group;
            for (int tok = 0; tok < held && tok <= qpos; ++tok) {
                int times = 0;
                bool inner = false;
                for (int v = 0; v < t.blks; ++v) {
                    const int tok0 = tile_block(t, v) * kBlock;
                    if (tok < tok0 || tok >= tok0 + kBlock) continue;
                    ++times;
                    inner = block_inner(t, tok0, kBlock, sinks);
                }
                const bool seen = key_seen(tok, qpos, window_low(qpos, window), sinks);
                if (times > 1 || (seen && times != 1) || (inner && !seen)) return GPTQ_ECHECK;
            }
        }
        for (int v = 0; v < t.blks; ++v) {
            const int tok0 = tile_block(t, v) * kBlock;
            if (tok0 < 0 || tok0 >= held) return GPTQ_ECHECK;
            if (block_inner(t, tok0, kBlock, sinks) && tok0 + kBlock > t.pos0 + x0 / group + 1) return GPTQ_ECHECK;
        }
    }
    return GPTQ_OK;
}
