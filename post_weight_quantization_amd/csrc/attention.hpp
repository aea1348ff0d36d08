// attention.hpp -- what the kernels that look at cached keys and values share (attention.hip, score.hip):
// arguments, a call's tiles and blocks, pages, and codes as matrix operands.
#pragma once
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

inline bool qheads_ok(const gptq_cache* c, int qheads) {
    return qheads >= c->heads && qheads % c->heads == 0 && qheads / c->heads <= 64;
}

}  // namespace gptq
