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
// attention_rows_kernel serves few rows to a sequence, attention_tile_kernel many; attn_plan chooses and
// cuts sequences into pieces, which attention_join_kernel adds in a fixed order.
#include <math.h>

#include <type_traits>

#include "../../include/gptq_check.h"
#include "cache.hpp"

namespace gptq {

struct AttnArgs {
    CacheView c;
    Batch q;
    const void* Q;
    int64_t ldq, ldqh;
    int qheads, group;
    float scale2;  // |scale| times log2 e: the softmax runs on powers of two
    uint32_t flip; // sign of scale, for Q's terms: 0 or two bf16 sign bits
    int window, sinks;
    void* O;
    int64_t ldo, ldoh;
    float* lse;
    float* part;     // [splits][rows][qheads][dim], then [splits][rows][qheads] of (maximum, sum)
    int splits;
    uint32_t page_m;  // page_div
    int page_shift;
};

// Division by d = page / 16 (up to 2^16) as a product: with 2^b >= d, m = ceil(2^(26 + b) / d) and n < 2^26,
// n m >> 26 + b = floor(n / d), since m d - 2^(26 + b) < d <= 2^b.  A sequence's n, tokens / 16, stay below.
struct PageDiv {
    uint32_t m;
    int shift;
};
inline PageDiv page_div(int page) {
    const uint32_t d = (uint32_t)page / 16;
    int b = 0;
    while ((1u << b) < d) ++b;
    return PageDiv{(uint32_t)(((1ull << (26 + b)) + d - 1) / d), 26 + b};
}

constexpr int kAttnWaves = 4;
constexpr int kBlock = 32;      // tokens a wave takes at a time
constexpr int kRowsTile = 16;   // query rows of a workgroup
constexpr int kMinBlocks = 8;   // blocks of a piece at least

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
                                                     int rows_tile, int block, Tile& t) {
    L = L > 0 ? L : 0;
    t.pos0 = L - t.R;
    const int q0 = t.x0 / group, last = (t.x0 + rows_tile - 1) / group, q1 = last < t.R - 1 ? last : t.R - 1;
    const int64_t end = (int64_t)t.pos0 + q1 + 1 < held ? (int64_t)t.pos0 + q1 + 1 : held;
    t.end = end > 0 ? (int)end : 0;
    const int64_t low = window ? (int64_t)t.pos0 + q0 - window + 1 : 0;
    t.lo_blk = low > 0 ? (int)(low / block) : 0;
    const int end_blk = (int)(((int64_t)t.end + block - 1) / block);
    const int before = t.lo_blk < end_blk ? t.lo_blk : end_blk;
    const int sink = window ? (int)(((int64_t)sinks + block - 1) / block) : 0;
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
__device__ __forceinline__ void tile_of_call(const AttnArgs& a, int rows_tile, int block, Tile& t) {
    tile_blocks(a.q.len[t.b], (int64_t)a.q.width * a.c.page, a.group, a.window, a.sinks, rows_tile, block, t);
}

// Grid: x the kv heads and, behind them, the pieces; y and z the tiles.  The tiles that the call's sizes
// allow but its sequences do not fill come last then: in between, where tiles ran along x, they left
// shader engines with a workgroup too many (4 x 256 rows over 8192 tokens in two pieces: 375 us).
constexpr int kGridTiles = 1 << 15;

__device__ __forceinline__ int tiles_of(int rows, int group, int rows_tile) {
    return (int)(((int64_t)rows * group + rows_tile - 1) / rows_tile);
}
// Up to kPacked sequences are counted through, and their tiles follow each other.  With more, the first
// tile of sequence b is tile start[b] group / rows_tile + b of the grid (rounded down), which leaves room for
// all of b's and is looked for in few steps: counted through, 20000 single rows took 22 us a workgroup.
constexpr int kPacked = 64;

// The tile of a workgroup: sequences in order, a sequence's last rows, which see the most tokens, first.
// What it finds is the same in every lane, and handed out in scalar registers.
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int rows_tile, Tile& t) {
    const int x = blockIdx.y + blockIdx.z * kGridTiles;
    if (!a.q.start) {
        const int per = (a.group + rows_tile - 1) / rows_tile;
        t.b = x / per;
        t.r0 = t.b;
        t.R = 1;
        t.x0 = (x - t.b * per) * rows_tile;
        return t.b < a.q.seqs;
    }
    const int lane = threadIdx.x & 63;
    if (a.q.seqs <= kPacked) {
        int r0 = 0, r1 = 0;
        if (lane < a.q.seqs) seq_rows(a.q, lane, r0, r1);
        int sum = tiles_of(r1 - r0, a.group, rows_tile);
#pragma unroll
        for (int k = 1; k < 64; k *= 2) {
            const int y = __shfl_up(sum, k);
            if (lane >= k) sum += y;
        }
        const unsigned long long past = __ballot(sum > x);
        if (!past) return false;
        const int l = __builtin_ctzll(past);
        t.b = l;
        t.r0 = __builtin_amdgcn_readlane(r0, l);
        t.R = __builtin_amdgcn_readlane(r1, l) - t.r0;
        t.x0 = (__builtin_amdgcn_readlane(sum, l) - 1 - x) * rows_tile;
        return true;
    }
    auto first = [&](int b) {
        int r0, r1;
        seq_rows(a.q, b, r0, r1);
        return (int)((int64_t)r0 * a.group / rows_tile) + b;
    };
    t.b = last_at_most(a.q.seqs, x, first);
    if (t.b < 0) return false;
    int r0, r1;
    seq_rows(a.q, t.b, r0, r1);
    t.r0 = __builtin_amdgcn_readfirstlane(r0);
    t.R = __builtin_amdgcn_readfirstlane(r1) - t.r0;
    const int at = tiles_of(t.R, a.group, rows_tile) - 1 - (x - first(t.b));
    t.x0 = at * rows_tile;
    return at >= 0 && t.x0 < t.R * a.group;  // the second always, where starts ascend
}

// Where the 16 tokens from `tok` (a multiple of 16) on are kept: the cache row of the first, on page 0
// where they have none, and whether they have.
__device__ __forceinline__ int64_t find_page(const AttnArgs& a, const int32_t* table, int head, int tok, bool& there) {
    const uint32_t n = (uint32_t)tok >> 4;
    const uint32_t at = (uint32_t)((uint64_t)n * a.page_m >> a.page_shift);  // n / (page / 16)
    const int page = (int)at < a.q.width ? table[at] : -1;
    there = (unsigned)page < (unsigned)a.c.pages;
    return ((int64_t)(there ? page : 0) * a.c.heads + head) * a.c.page + (tok - (int)at * a.c.page);
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
// The G scales of four tokens in a row, as they lie, and scale i of token r of them.
template <int G>
__device__ __forceinline__ void load_scales(const uint16_t* p, uint32_t (&w)[2 * G]) {
#pragma unroll
    for (int k = 0; k < G / 2; ++k) {
        const u32v4 v = ((const u32v4*)p)[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * k + j] = v[j];
    }
}
template <int G>
__device__ __forceinline__ float scale_of(const uint32_t (&w)[2 * G], int r, int i) {
    const uint32_t x = w[(r * G + i) >> 1];
    return __uint_as_float((i & 1) ? x & 0xffff0000u : x << 16);
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

// The nibbles of x at even or odd places, a byte each.  The empty statement hides the mask: seeing it, the
// compiler takes every byte out by a field extract of its own before it converts it.
__device__ __forceinline__ uint32_t nibble_bytes(uint32_t x, bool odd) {
    uint32_t y = (odd ? x >> 4 : x) & 0x0f0f0f0fu;
    asm("" : "+v"(y));
    return y;
}
// Codes in two registers' bytes times s, exact in bf16: (low half <- byte LO of y, high half <- byte HI).
template <int LO, int HI>
__device__ __forceinline__ uint32_t decode_pair(uint32_t y, float s0, float o0, float s1, float o1) {
    const float a = fmaf((float)(y >> (8 * LO) & 255u), s0, o0), b = fmaf((float)(y >> (8 * HI) & 255u), s1, o1);
    return pack_hi(__float_as_uint(a), __float_as_uint(b));
}

// Key word w as an operand: its codes as 16 + code + 8, or, in f32, as they are.  The offset costs f32 sums
// a few bits (24 against codes up to 7), which only f32 has use for; without it the unpacking takes three
// times the instructions.
template <int DT>
__device__ __forceinline__ u32v4 key_operand(uint32_t w) {
    if constexpr (DT != GPTQ_F32) {
        return unpack_nibbles(w);
    } else {
        const uint32_t even = nibble_bytes(w, false), odd = nibble_bytes(w, true);
        return u32v4{decode_pair<0, 2>(even, 1.0f, -8.0f, 1.0f, -8.0f), decode_pair<0, 2>(odd, 1.0f, -8.0f, 1.0f, -8.0f),
                     decode_pair<1, 3>(even, 1.0f, -8.0f, 1.0f, -8.0f), decode_pair<1, 3>(odd, 1.0f, -8.0f, 1.0f, -8.0f)};
    }
}
// The same for nibble N of the halves of x (two tokens).
template <int DT, int N>
__device__ __forceinline__ uint32_t value_operand(uint32_t x) {
    if constexpr (DT != GPTQ_F32) {
        return nibble_pair<N>(x);
    } else {
        const uint32_t y = nibble_bytes(x, N & 1);
        return N < 2 ? decode_pair<0, 2>(y, 1.0f, -8.0f, 1.0f, -8.0f) : decode_pair<1, 3>(y, 1.0f, -8.0f, 1.0f, -8.0f);
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

// attention_rows_kernel: a workgroup owns 16 query rows (the query heads of one kv head, times the rows of
// one sequence) and a piece of the sequence; its four waves take 32 tokens at a time and are joined in
// LDS.  A block's instructions (380 vector ones at dim 128: unpacking, scales to scores and weights,
// exponentials) are shared by 16 rows only, so beside the read of the codes they bound it: 64 sequences of
// up to 4096 tokens, 8 heads of 8 queries, take 61 us, 3.5 TB/s of cache; vector instructions are in 47 % of
// a SIMD's cycles then and MFMA in 9 %, by the hardware's counters.
template <int DT, int G>
__global__ __launch_bounds__(kAttnWaves * 64, G == 2 ? 3 : G == 8 ? 1 : 2) void attention_rows_kernel(AttnArgs a) {
    constexpr int NT = kTerms<DT>;
    constexpr int D = 32 * G;
    // Blocks on their way that registers hold without spills.  Two at dim 128 in bf16 spilled 9 of them and took
    // longer at every size (64 x 4096 tokens of 8 x 8 heads 73 us against 68, 1500 of 8 x 4 12.5 against 11.7).
    constexpr int AHEAD = G == 2 ? 2 : 1;
    __shared__ float joined[kAttnWaves][2 * G][64][4];
    __shared__ float stat[kAttnWaves][2][16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int split = blockIdx.x / a.c.heads, head = blockIdx.x - split * a.c.heads;
    Tile t;
    if (!find_tile(a, kRowsTile, t)) return;
    tile_of_call(a, kRowsTile, kBlock, t);
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
#pragma unroll
        for (int k = 0; k < NT; ++k) q[i][k] ^= a.flip;
        start[i] = f32v4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NT; ++k)
            if constexpr (DT != GPTQ_F32) start[i] = mfma16(minus24, q[i][k], start[i]);
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
    // A block as it is loaded: keys, values and their scales of two 16-token tiles.  Up to two blocks are on
    // their way; a block's keys make place for those of a later one as soon as they are multiplied, its
    // values likewise.  Addresses are a place that is the same in the wave plus a lane's constant offset.
    struct Block {
        uint32_t kw[2][G], ks[2][2 * G], vw[2][4][(G + 3) / 4], vs[2][2 * G];
        bool there[2];
    };
    int64_t place[2];
    bool coming[2];
    const uint32_t klane = c * (16 * G) + h * (4 * G), vlane = 4 * h * (16 * G) + c * G, slane = 4 * h * G;
    auto find = [&](int v) {
        const int tok0 = tile_block(t, v) * kBlock;
#pragma unroll
        for (int u = 0; u < 2; ++u) place[u] = find_page(a, table, head, tok0 + 16 * u, coming[u]);
    };
    auto fetch_keys = [&](Block& k) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            load_key_words<G>(a.c.k + place[u] * (16 * G) + klane, k.kw[u]);
            load_scales<G>(a.c.ks + place[u] * G + slane, k.ks[u]);
        }
    };
    auto fetch_values = [&](Block& k) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                load_value_words<G>(a.c.v + place[u] * (16 * G) + vlane + r * (16 * G), k.vw[u][r]);
            load_scales<G>(a.c.vs + place[u] * G + slane, k.vs[u]);
            k.there[u] = coming[u];
        }
    };
    auto turn = [&](int v, Block& now) {
        const int tok0 = tile_block(t, v) * kBlock;
        find(min(v + AHEAD * kAttnWaves, v1 - 1));  // behind the end the last block again
        float p[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f32v4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const u32v4 kk = key_operand<DT>(now.kw[u][i]);
                f32v4 d = start[i];
#pragma unroll
                for (int k = 0; k < NT; ++k) d = mfma16(kk, q[i][k], d);
#pragma unroll
                for (int r = 0; r < 4; ++r) s[r] = fmaf(scale_of<G>(now.ks[u], r, i), d[r], s[r]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) p[4 * u + r] = s[r];
        }
        fetch_keys(now);
        // Blocks at an edge of what the rows see (or with an absent page): score by score.  Selects, not
        // branches around the assignments: under branches the compiler keeps the unmasked scores.
        const bool inner = now.there[0] && now.there[1] && block_inner(t, tok0, kBlock, a.sinks);
        if (!inner) {
            // Bounds from this lane's first token on; the empty statement keeps them in here.
            int first = tok0 + 4 * h;
            asm("" : "+v"(first));
            const int to = qpos - first, from = low - first, sinks = a.sinks - first;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = 16 * (j >> 2) + (j & 3);
                const bool seen = now.there[j >> 2] & (k <= to) & ((k > from) | (k < sinks));
                p[j] = seen ? p[j] : -INFINITY;
                // A hidden token's scales may be anything: 0 times them is not 0.
                const uint32_t keep = seen ? ~0u : 0u;
                if constexpr (G == 2) {
                    now.vs[j >> 2][j & 3] &= keep;
                } else {
#pragma unroll
                    for (int i = 0; i < G / 2; ++i) now.vs[j >> 2][(j & 3) * (G / 2) + i] &= keep;
                }
            }
        }
        float top = p[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = fmaxf(top, p[j]);
        top = fmaxf(m, quad_max(top) * a.scale2);
        // The sums move to a new maximum only when one has risen by 8 (weights up to 2^8 are harmless).
        if (__ballot(top > m + 8.0f)) {
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
        const float base = m == -INFINITY ? 0.0f : -m;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] = __builtin_amdgcn_exp2f(fmaf(p[j], a.scale2, base));
            l += p[j];
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            // Weights times the group's scales.
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = p[j] * scale_of<G>(now.vs[j >> 2], j & 3, i);
            u32v4 pt[NT];
            weight_terms<DT>(w, pt);
#pragma unroll
            for (int k = 0; k < NT; ++k)
                if constexpr (DT != GPTQ_F32) fix[i] = mfma16(minus24, pt[k], fix[i]);
            // Codes of group i, channels m and 16 + m: nibbles 2 (i % 2) and the next of half i / 2.
            u32v4 c0, c1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int u = k >> 1, r = 2 * (k & 1), word = i >> 2;
                const uint32_t x = (i >> 1 & 1) ? pack_hi(now.vw[u][r][word], now.vw[u][r + 1][word])
                                                : pack_lo(now.vw[u][r][word], now.vw[u][r + 1][word]);
                c0[k] = (i & 1) ? value_operand<DT, 2>(x) : value_operand<DT, 0>(x);
                c1[k] = (i & 1) ? value_operand<DT, 3>(x) : value_operand<DT, 1>(x);
            }
#pragma unroll
            for (int k = 0; k < NT; ++k) {
                o[i][0] = mfma16(c0, pt[k], o[i][0]);
                o[i][1] = mfma16(c1, pt[k], o[i][1]);
            }
        }
        fetch_values(now);
    };
    Block even, odd;
    if (v0 + wave < v1) {
        find(v0 + wave);
        fetch_keys(even);
        fetch_values(even);
        if constexpr (AHEAD == 2) {
            find(min(v0 + wave + kAttnWaves, v1 - 1));
            fetch_keys(odd);
            fetch_values(odd);
        }
    }
    for (int v = v0 + wave; v < v1; v += AHEAD * kAttnWaves) {
        turn(v, even);
        if constexpr (AHEAD == 2)
            if (v + kAttnWaves < v1) turn(v + kAttnWaves, odd);
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

// attention_tile_kernel: many rows to a sequence.  A workgroup owns 128 NQ query rows of one kv head (16 NQ
// a wave) and walks the tokens 64 at a time.  The tile's keys and values are decoded once, to bf16,
// where c s is exact, straight into operand order in LDS, and all eight waves read them from there; the
// scales are in the operands, so a score is one accumulator and a softmax weight one operand.  The next
// tile's codes are on their way meanwhile.  Waves 0 to 3 decode the keys of 16 tokens each, waves 4 to 7
// half the channels of the values of 32: one of either kind on each SIMD.
//
// Bound by the vector instructions of the softmax and the decoding and by the waits between them and MFMA: 2 x
// up to 2048 rows of 16 heads over 8192 tokens take 270 us, 560 TFLOP/s, with vector instructions in 50 %
// of a SIMD's cycles and MFMA in 24 %, by the hardware's counters, and 33 us to join the pieces.
//
// In a tile that not every row sees all of, a value group whose scale is not finite enters LDS as zeros
// and its token is marked; rows that see it get NaN there, others do not (a weight of 0 times NaN would
// reach them).
constexpr int kTokens = 64, kAttnTileWaves = 8;

template <int DT, int G>
constexpr int kQTiles = G * kTerms<DT> <= 8 && G <= 4 ? 2 : 1;  // what 256 registers hold, but for few spills

template <int DT, int G>
__global__ __launch_bounds__(kAttnTileWaves * 64) void attention_tile_kernel(AttnArgs a) {
    constexpr int NT = kTerms<DT>, NQ = kQTiles<DT, G>, ROWS = kAttnTileWaves * 16 * NQ, D = 32 * G;
    // Registers of queries, sums and weights.  Where they are half of the 256, operands are read from LDS as
    // they are used, not ahead, and values loaded just before they are decoded, not a turn earlier: that spills
    // fewer registers.  Spilled, and us at 4 x 512 rows of 32 heads over 4096 tokens, otherwise -> so:
    //   f32   dim 256 249, 1985 -> 28, 674    dim 128 none, 377 -> none, 377    dim 64 29, 248 -> none, 229
    //   f16   dim 256 137, 1080 -> none, 517  dim 128 70, 321 -> 27, 250        dim 64 none either way
    // and the two that keep the reads ahead, spilling less than they would wait: bf16 dim 256 19, 392 (none, 433
    // so), dim 128 one, 185 (none, 194).  The build fails where more are spilled than it names.
    constexpr bool TIGHT = NQ * (4 * G * NT + 8 * G + 8 * NT) >= 128;
    constexpr int DEEP = TIGHT ? 1 : 2;
    __shared__ u32v4 ks[2][4][G][64];
    __shared__ u32v4 vs[2][2][G][2][64];
    __shared__ unsigned long long bad[3][G];  // marked tokens of each group of the values, three tiles' turns
    __shared__ uint32_t there[2];             // a byte for each 16 tokens: 1 where their page exists
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, h = lane >> 4;
    const int split = blockIdx.x / a.c.heads, head = blockIdx.x - split * a.c.heads;
    Tile t;
    if (!find_tile(a, ROWS, t)) return;
    tile_of_call(a, ROWS, kTokens, t);
    const int per = piece_blocks(t.blks, a.splits);
    const int v0 = split * per, v1 = min(t.blks, v0 + per);
    if (v0 >= v1 && split != 0) return;
    const bool whole = t.blks <= per;

    int qi[NQ], qh[NQ], qpos[NQ], low[NQ];
    u32v4 q[NQ][G][NT];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int x = min(t.x0 + (wave * NQ + n) * 16 + c, t.R * a.group - 1);
        qi[n] = x / a.group;
        qh[n] = head * a.group + (x - qi[n] * a.group);
        qpos[n] = t.pos0 + qi[n];
        low[n] = window_low(qpos[n], a.window);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            load_terms<DT, false>(a.Q, (int64_t)(t.r0 + qi[n]) * a.ldq + (int64_t)qh[n] * a.ldqh + 32 * i + 8 * h, q[n][i]);
#pragma unroll
            for (int k = 0; k < NT; ++k) q[n][i][k] ^= a.flip;
        }
    }
    f32v4 o[NQ][G][2];
    float m[NQ], l[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        m[n] = -INFINITY;
        l[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i) o[n][i][0] = o[n][i][1] = f32v4{0.f, 0.f, 0.f, 0.f};
    }

    // This wave's part of a tile, as it is loaded: the words of a key and its scales, or of eight tokens'
    // values (half `vi` of the channels of tokens 32 vb ..) and theirs.
    const bool keys = wave < 4;
    const int vb = wave >> 1 & 1, vi = wave & 1;
    const int32_t* table = a.q.table + (int64_t)t.b * a.q.width;
    constexpr int VW = (G + 3) / 4;
    uint32_t raw[8 * VW + 4 * G];
    bool there0 = false, there1 = false, edge = false;
    int vtok = 0;
    auto fetch = [&](int v) {
        const int tok0 = tile_block(t, v) * kTokens;
        if (keys) {
            const int64_t p = find_page(a, table, head, tok0 + 16 * wave, there0);
            uint32_t w[G];
            load_key_words<G>(a.c.k + (p + c) * (16 * G) + h * (4 * G), w);
            const uint32_t* sp = (const uint32_t*)(a.c.ks + (p + c) * G);
#pragma unroll
            for (int i = 0; i < G; ++i) raw[i] = w[i];
#pragma unroll
            for (int i = 0; i < G / 2; ++i) raw[G + i] = sp[i];
        } else {
            vtok = tok0 + 32 * vb;
            const int64_t p0 = find_page(a, table, head, vtok, there0), p1 = find_page(a, table, head, vtok + 16, there1);
            edge = !(there0 & there1 & block_inner(t, tok0, kTokens, a.sinks));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t p = (u ? p1 : p0) + 4 * h;
                uint32_t w[VW], sc[2 * G];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    load_value_words<G>(a.c.v + (p + r) * (16 * G) + c * G, w);
#pragma unroll
                    for (int k = 0; k < VW; ++k) raw[(4 * u + r) * VW + k] = w[k];
                }
                load_scales<G>(a.c.vs + p * G, sc);
#pragma unroll
                for (int k = 0; k < 2 * G; ++k) raw[8 * VW + 2 * G * u + k] = sc[k];
            }
        }
    };
    // Scale i of token 4 h + r of the 16 tokens u.
    auto vscale = [&](int u, int r, int i) {
        const uint32_t x = raw[8 * VW + 2 * G * u + ((r * G + i) >> 1)];
        return __uint_as_float((i & 1) ? x & 0xffff0000u : x << 16);
    };
    auto values = [&](auto masked, int buf, int turn) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            unsigned long long mark = 0ull;
            u32v4 w;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    float s[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        s[e] = vscale(u, r + e, i);
                        if constexpr (decltype(masked)::value) {
                            const int tok = 16 * u + 4 * h + r + e;
                            const bool live = (u ? there1 : there0) && vtok + tok < t.end;  // others hold anything
                            const bool odd = (__float_as_uint(s[e]) & 0x7f800000u) == 0x7f800000u;
                            mark |= live && odd ? 1ull << (32 * vb + tok) : 0ull;
                            s[e] = live && !odd ? s[e] : 0.0f;
                        }
                    }
                    const uint32_t a0 = raw[(4 * u + r) * VW + (i >> 2)], a1 = raw[(4 * u + r + 1) * VW + (i >> 2)];
                    const uint32_t x = (i >> 1 & 1) ? pack_hi(a0, a1) : pack_lo(a0, a1);
                    const uint32_t y = nibble_bytes(x, vi);
                    const float z0 = -8.0f * s[0], z1 = -8.0f * s[1];
                    w[2 * u + (r >> 1)] = (i & 1) ? decode_pair<1, 3>(y, s[0], z0, s[1], z1)
                                                  : decode_pair<0, 2>(y, s[0], z0, s[1], z1);
                }
            vs[buf][vb][i][vi][lane] = w;
            // Every lane of a quarter has the same marks; both halves of the channels do.
            if constexpr (decltype(masked)::value)
                if (vi == 0 && c == 0 && mark) atomicOr(&bad[turn][i], mark);
        }
    };
    auto decode = [&](int buf, int turn) {
        if (keys) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const uint32_t x = raw[G + (i >> 1)];
                const float s = __uint_as_float((i & 1) ? x & 0xffff0000u : x << 16), z = -8.0f * s;
                const uint32_t even = nibble_bytes(raw[i], false), odd = nibble_bytes(raw[i], true);
                ks[buf][wave][i][lane] = u32v4{decode_pair<0, 2>(even, s, z, s, z), decode_pair<0, 2>(odd, s, z, s, z),
                                               decode_pair<1, 3>(even, s, z, s, z), decode_pair<1, 3>(odd, s, z, s, z)};
            }
            if (lane == 0) ((uint8_t*)&there[buf])[wave] = there0 ? 1 : 0;
        } else if (edge) {
            values(std::true_type{}, buf, turn);
        } else {
            values(std::false_type{}, buf, turn);
        }
    };

    if (threadIdx.x < 3 * G) bad[threadIdx.x / G][threadIdx.x % G] = 0ull;
    __syncthreads();
    if (v0 < v1) {
        fetch(v0);
        decode(0, 0);
        if (!keys && !TIGHT) fetch(min(v0 + 1, v1 - 1));
    }
    __syncthreads();
    int turn = 0;
    int buf = 0;
    for (int v = v0; v < v1; ++v) {
        // The two kinds of waves decode the next tile at opposite ends of the turn, so that on a SIMD one
        // multiplies while the other decodes or takes exponentials.  The marks of the tile before were
        // read by all before the last barrier; they are set again behind the next one.
        const int next = turn == 2 ? 0 : turn + 1;
        if (threadIdx.x < G) bad[next == 2 ? 0 : next + 1][threadIdx.x] = 0ull;
        if (keys) {
            fetch(min(v + 1, v1 - 1));
        } else {
            if (TIGHT) fetch(min(v + 1, v1 - 1));
            decode(buf ^ 1, next);
            if (!TIGHT) fetch(min(v + 2, v1 - 1));
        }
        const int tok0 = tile_block(t, v) * kTokens;
        // Keys of the next 16 tokens are read while those of these are multiplied.
        f32v4 s[NQ][4];
        u32v4 kk[DEEP][G];
#pragma unroll
        for (int i = 0; i < G; ++i) kk[0][i] = ks[buf][0][i][lane];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (DEEP == 1 && u > 0) {
#pragma unroll
                for (int i = 0; i < G; ++i) kk[0][i] = ks[buf][u][i][lane];
            }
            if (DEEP == 2 && u < 3) {
#pragma unroll
                for (int i = 0; i < G; ++i) kk[(u + 1) % DEEP][i] = ks[buf][u + 1][i][lane];
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < NT; ++e)
                        s[n][u] = mfma16(kk[u % DEEP][i], q[n][i][e], i + e == 0 ? f32v4{0.f, 0.f, 0.f, 0.f} : s[n][u]);
        }
        const uint32_t exist = __builtin_amdgcn_readfirstlane(there[buf]);
        const bool inner = exist == 0x01010101u && block_inner(t, tok0, kTokens, a.sinks);
        u32v4 pt[NQ][2][NT];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float p[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = s[n][j >> 2][j & 3];
            if (!inner) {
                // Bounds from this lane's first token on; the empty statement keeps them in here.
                int first = tok0 + 4 * h;
                asm("" : "+v"(first));
                const int to = qpos[n] - first, from = low[n] - first, sinks = a.sinks - first;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int k = 16 * (j >> 2) + (j & 3);
                    const bool seen = (exist >> (8 * (j >> 2)) & 1u) & (k <= to) & ((k > from) | (k < sinks));
                    p[j] = seen ? p[j] : -INFINITY;
                }
            }
            float top = p[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) top = fmaxf(top, p[j]);
            top = fmaxf(m[n], quad_max(top) * a.scale2);
            // The sums move to a new maximum only when one has risen by 8 (weights up to 2^8 are harmless).
            if (__ballot(top > m[n] + 8.0f)) {
                const float less = m[n] == top ? 1.0f : exp2f(m[n] - top);
                m[n] = top;
                l[n] *= less;
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        o[n][i][0][r] *= less;
                        o[n][i][1][r] *= less;
                    }
            }
            const float base = m[n] == -INFINITY ? 0.0f : -m[n];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                p[j] = __builtin_amdgcn_exp2f(fmaf(p[j], a.scale2, base));
                l[n] += p[j];
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = p[8 * b + j];
                weight_terms<DT>(w, pt[n][b]);
            }
        }
        // Values two groups at a time, the next two on their way.
        constexpr int VB = 4 * G;  // operands of the tile's values
        u32v4 vv[DEEP][4];
        auto value = [&](int k) { return vs[buf][k / (2 * G)][k / 2 % G][k & 1][lane]; };
#pragma unroll
        for (int k = 0; k < 4; ++k) vv[0][k] = value(k);
#pragma unroll
        for (int k0 = 0; k0 < VB; k0 += 4) {
            if (DEEP == 1 && k0 > 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) vv[0][k] = value(k0 + k);
            }
            if (DEEP == 2 && k0 + 4 < VB) {
#pragma unroll
                for (int k = 0; k < 4; ++k) vv[((k0 >> 2) + 1) % DEEP][k] = value(k0 + 4 + k);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int b = (k0 + k) / (2 * G), i = (k0 + k) / 2 % G, f = k & 1;
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < NT; ++e) o[n][i][f] = mfma16(vv[(k0 >> 2) % DEEP][k], pt[n][b][e], o[n][i][f]);
            }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            if (inner) break;
            const unsigned long long marks = bad[turn][i];
            if (marks == 0ull) continue;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                bool sees = false;
#pragma unroll 1
                for (int j = 0; j < kTokens; ++j)
                    if (marks >> j & 1ull) sees |= key_seen(tok0 + j, qpos[n], low[n], a.sinks);
                const float add = sees ? __uint_as_float(0x7fc00000u) : 0.0f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    o[n][i][0][r] += add;
                    o[n][i][1][r] += add;
                }
            }
        }
        if (keys) decode(buf ^ 1, next);
        __syncthreads();
        buf ^= 1;
        turn = next;
    }

#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const float sum = quad_sum(l[n]);
        if (t.x0 + (wave * NQ + n) * 16 + c >= t.R * a.group) continue;
        const int64_t row = t.r0 + qi[n], item = row * a.qheads + qh[n];
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int d = 32 * i + 16 * f + 4 * h;
                if (whole) {
                    float y[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[r] = o[n][i][f][r] * inv;
                    store_four<DT>(a.O, row * a.ldo + (int64_t)qh[n] * a.ldoh + d, y);
                } else {
                    *(f32v4*)(a.part + ((int64_t)split * a.q.rows * a.qheads + item) * D + d) = o[n][i][f];
                }
            }
        if (h == 0) {
            if (!whole) {
                float* ml = a.part + (int64_t)a.splits * a.q.rows * a.qheads * D +
                            2 * ((int64_t)split * a.q.rows * a.qheads + item);
                ml[0] = m[n];
                ml[1] = sum;
            } else if (a.lse) {
                a.lse[item] = sum == 0.0f ? -INFINITY : (m[n] + log2f(sum)) * 0.69314718055994531f;
            }
        }
    }
}

// One wave per row and query head (of a kernel with tiles of rows_tile rows and blocks of `block`
// tokens): the pieces' sums over a common maximum, in order.  Bound by their read (and a launch).
template <int DT, int G>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int rows_tile, int block) {
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
    t.x0 = ((row - t.r0) * a.group + qh % a.group) / rows_tile * rows_tile;
    tile_of_call(a, rows_tile, block, t);
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
typedef void (*JoinKernel)(AttnArgs, int, int);
struct AttnPick {
    AttnKernel rows, tile;
    JoinKernel join;
};
template <int DT>
static AttnPick attn_kernels(int dim) {
    if (dim == 64) return {attention_rows_kernel<DT, 2>, attention_tile_kernel<DT, 2>, attention_join_kernel<DT, 2>};
    if (dim == 128) return {attention_rows_kernel<DT, 4>, attention_tile_kernel<DT, 4>, attention_join_kernel<DT, 4>};
    return {attention_rows_kernel<DT, 8>, attention_tile_kernel<DT, 8>, attention_join_kernel<DT, 8>};
}
// Query rows of attention_tile_kernel's workgroup.
static int attn_tile_rows(int dtype, int dim) {
    const int g = dim / 32, nt = dtype == GPTQ_BF16 ? 1 : dtype == GPTQ_F16 ? 2 : 3;
    return kAttnTileWaves * 16 * (g * nt <= 8 && g <= 4 ? 2 : 1);
}

// Tiles of rows_tile query rows of one kv head, at most: each sequence may end in a part of one.
static int64_t tiles_at_most(const gptq_batch* b, int group, int rows_tile) {
    if (!b->start) return (int64_t)b->seqs * ((group + rows_tile - 1) / rows_tile);
    const int64_t most = (b->rows * group + rows_tile - 1) / rows_tile + b->seqs;
    return b->seqs > kPacked || most < b->rows * group ? most : b->rows * group;
}
// How a call is cut: which kernel, its tile of query rows, its blocks of tokens, the pieces of a sequence.
struct AttnPlan {
    bool tile;
    int rows_tile, block, splits;
};
static AttnPlan attn_plan(const gptq_cache* c, const gptq_batch* b, int group, int dtype) {
    AttnPlan p;
    // Rows of an average sequence (the lengths are on the device).
    p.tile = b->rows * group >= 64 * (int64_t)b->seqs;
    p.rows_tile = p.tile ? attn_tile_rows(dtype, c->dim) : kRowsTile;
    p.block = p.tile ? kTokens : kBlock;
    // Pieces a sequence is cut into.  What a call takes is taken to be the rounds of workgroups that the CUs
    // hold, times the turns of a piece (of the longest sequence the table can hold) and what a piece
    // costs beside them, its sums written and joined: about 6 turns of the tile kernel (64 tokens), 4 of the
    // rows kernel (128).  More pieces are taken where that saves a tenth, and none where there
    // is a round without; a piece keeps kMinBlocks blocks.
    // Measured (us, bf16, 8 heads, dim 128; pieces taken in brackets):
    //   4 x 256 rows of 32 heads over 8192 tokens    1: 353, [2: 215], 3: 278, 4: 225, 8: 252
    //   512 rows of 32 heads over 4096 tokens        1: 186, 3: 95, [4: 78], 6: 106, 8: 92
    //   2048 rows of 32 heads over 2048 tokens      [1: 102], 2: 123, 4: 164
    //   16 x 1 row of 32 heads over 8192 tokens      1: 82, 2: 51, [4: 42], 8: 46, 16: 53
    //   64 x 1 row of 64 heads over 4096 tokens     [1: 71], 2: 76, 4: 80
    //   200 x 1 row of 64 heads, up to 2048 tokens  [1: 95], 2: 106, 3: 111
    // One kernel and one number of pieces serve the whole call: 63 single rows beside 2048 rows of one sequence (32
    // heads on 8 of 128, 4096 tokens each) take 550 us on the tile kernel, in two calls 67 and 185.
    const int64_t each = b->start ? (b->rows + b->seqs - 1) / b->seqs : 1;  // rows of an average sequence
    const int64_t even = b->seqs * ((each * group + p.rows_tile - 1) / p.rows_tile);
    const int64_t most_tiles = tiles_at_most(b, group, p.rows_tile);
    const int64_t wg = (even < most_tiles ? even : most_tiles) * c->heads;
    const int64_t hold = kCUs * (p.tile ? 1 : c->dim == 64 ? 3 : c->dim == 256 ? 1 : 2);
    const int64_t blks = ((int64_t)b->width * c->page + p.block - 1) / p.block;
    const int64_t most = (blks + kMinBlocks - 1) / kMinBlocks;
    p.splits = 1;
    double best = 0.0;
    for (int64_t s = 1; s <= 64 && s <= most && (s == 1 || (wg < hold && (s - 1) * wg < 4 * hold)); ++s) {
        const int64_t per = piece_blocks((int)blks, (int)s);
        const double turns = p.tile ? (double)per : (double)(per / kAttnWaves);
        const double cost = (double)((s * wg + hold - 1) / hold) * (turns + (s > 1 || !p.tile ? (p.tile ? 6.0 : 4.0) : 0.0)) + 0.1 * (double)s;
        if (s == 1 || cost < 0.9 * best) {
            best = cost;
            p.splits = (int)s;
        }
    }
    return p;
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
                                                      int32_t q_heads, int dtype) {
    if (!cache || !batch_sizes_ok(batch) || !table_ok(cache, batch) || !dtype_size(dtype) || cache->heads < 1 || cache->page < 16 ||
        !(cache->dim == 64 || cache->dim == 128 || cache->dim == 256) || !qheads_ok(cache, q_heads))
        return 0;
    const int group = q_heads / cache->heads;
    return attn_part_bytes(cache, batch, q_heads, attn_plan(cache, batch, group, dtype).splits);
}

extern "C" int gptq_cache_attention(const gptq_cache* cache, const gptq_batch* batch, const void* Q, int64_t ldq,
                                    int64_t ldqh, int32_t q_heads, int dtype, float scale, int32_t window,
                                    int32_t sinks, void* O, int64_t ldo, int64_t ldoh, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    const int es = dtype_size(dtype);
    if (!es || !cache_ok(cache) || !batch_ok(batch) || !table_ok(cache, batch) || !qheads_ok(cache, q_heads)) return GPTQ_EINVAL;
    if (!isfinite(scale) || window < 0 || sinks < 0) return GPTQ_EINVAL;
    if (batch->rows == 0) return GPTQ_OK;
    if (!Q || !O || !heads_ok(Q, batch->rows, ldq, ldqh, q_heads, cache->dim, es) ||
        !heads_ok(O, batch->rows, ldo, ldoh, q_heads, cache->dim, es) || ((uintptr_t)lse & 3u))
        return GPTQ_EINVAL;
    // In place, a row's own workgroup reads it before any writes it: that needs the same strides.
    const bool in_place = O == Q && (batch->rows == 1 || ldo == ldq) && (q_heads == 1 || ldoh == ldqh);
    const RowSet o = heads_rows(O, batch->rows, ldo, ldoh, q_heads, cache->dim, es);
    if (!in_place && (O == Q || rows_meet(o, heads_rows(Q, batch->rows, ldq, ldqh, q_heads, cache->dim, es)))) return GPTQ_EINVAL;
    if (meets_cache(o, cache)) return GPTQ_EINVAL;
    const int group = q_heads / cache->heads;
    if (batch->rows * group > ((int64_t)1 << 27)) return GPTQ_EINVAL;
    const AttnPlan plan = attn_plan(cache, batch, group, dtype);
    int splits = plan.splits;
    if (window) {
        // Pieces that the window leaves without blocks are not launched (nor joined, if one is left: 8 rows of
        // 32 heads that see 128 of 4096 tokens 10.8 -> 8.0 us).
        const int64_t seen = ((int64_t)window + plan.rows_tile / group) / plan.block + 2 + ((int64_t)sinks + plan.block - 1) / plan.block;
        const int64_t most = (seen + kMinBlocks - 1) / kMinBlocks;
        if (splits > most) splits = (int)most;
    }
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
                     // above 0, so that hidden scores stay -inf, and finite
                     (float)fmin(fmax(fabs((double)scale) * 1.4426950408889634, 0x1p-100), 0x1p127),
                     scale < 0.0f ? 0x80008000u : 0u, window, sinks, O, ldo, ldoh, lse, (float*)workspace,
                     splits, page_div(cache->page).m, page_div(cache->page).shift};
    const AttnPick k = dtype == GPTQ_F32    ? attn_kernels<GPTQ_F32>(cache->dim)
                       : dtype == GPTQ_BF16 ? attn_kernels<GPTQ_BF16>(cache->dim)
                                            : attn_kernels<GPTQ_F16>(cache->dim);
    const AttnKernel run = plan.tile ? k.tile : k.rows;
    const int64_t tiles = tiles_at_most(batch, group, plan.rows_tile);
    const int64_t items = batch->rows * q_heads;
    const int64_t qw = (q_heads - 1) * ldqh + cache->dim, ow = (q_heads - 1) * ldoh + cache->dim;
    const int64_t pf = (int64_t)(need / 4);
    {
        ProfScope ps(FAM_ATTENTION, st, 0.0, 0.0);
        GPTQ_LAUNCH(st, plan.tile ? "attention_tile" : "attention_rows",
                    (run<<<dim3((unsigned)(cache->heads * splits), (unsigned)(tiles < kGridTiles ? tiles : kGridTiles),
                                (unsigned)((tiles + kGridTiles - 1) / kGridTiles)),
                           (plan.tile ? kAttnTileWaves : kAttnWaves) * 64, 0, st>>>(a)),
                    rd(Q, ldq, batch->rows, qw, es), batch_span(batch, 0), batch_span(batch, 1), batch_span(batch, 2),
                    plane(cache->k, cache, cache->dim / 2, false), plane(cache->v, cache, cache->dim / 2, false),
                    plane(cache->k_scale, cache, cache->dim / 16, false),
                    plane(cache->v_scale, cache, cache->dim / 16, false), wr(O, ldo, batch->rows, ow, es),
                    wr(lse ? (const void*)lse : O, items, lse ? 1 : 0, items),
                    wr(need ? (const void*)workspace : O, pf, need ? 1 : 0, pf));
        if (splits > 1)
            GPTQ_LAUNCH(st, "attention_join", (k.join<<<(unsigned)((items + 3) / 4), 256, 0, st>>>(a, plan.rows_tile, plan.block)),
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
                                           int32_t sinks, int32_t splits, int32_t rows_tile, int32_t block) {
    if (rows < 1 || group < 1 || held < 0 || window < 0 || sinks < 0 || splits < 1 || rows_tile < 1 || block < 1)
        return GPTQ_EINVAL;
    for (int x0 = 0; x0 < rows * group; x0 += rows_tile) {
        Tile t{};
        t.R = rows;
        t.x0 = x0;
        tile_blocks(len, held, group, window, sinks, rows_tile, block, t);
        const int per = piece_blocks(t.blks, splits);
        if ((int64_t)per * splits < t.blks || per % kAttnWaves) return GPTQ_ECHECK;
        for (int x = x0; x < x0 + rows_tile && x < rows * group; ++x) {
            const int qpos = t.pos0 + x / group;
            for (int tok = 0; tok < held && tok <= qpos; ++tok) {
                int times = 0;
                bool inner = false;
                for (int v = 0; v < t.blks; ++v) {
                    const int tok0 = tile_block(t, v) * block;
                    if (tok < tok0 || tok >= tok0 + block) continue;
                    ++times;
                    inner = block_inner(t, tok0, block, sinks);
                }
                const bool seen = key_seen(tok, qpos, window_low(qpos, window), sinks);
                if (times > 1 || (seen && times != 1) || (inner && !seen)) return GPTQ_ECHECK;
            }
        }
        for (int v = 0; v < t.blks; ++v) {
            const int tok0 = tile_block(t, v) * block;
            if (tok0 < 0 || tok0 >= held) return GPTQ_ECHECK;
            if (block_inner(t, tok0, block, sinks) && tok0 + block > t.pos0 + x0 / group + 1) return GPTQ_ECHECK;
        }
    }
    return GPTQ_OK;
}
