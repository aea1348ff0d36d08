// evict.hip -- cached tokens kept by their scores, on gfx950.
//
// Of each sequence and kv head: the first `sinks` tokens, the last `recent`, and of those between the highest
// scores, `keep` in all, moved together in their order.  evict_select_kernel finds them: the K-th largest score
// by its bits, 11 at a time from the top (a histogram in LDS, then its suffix sums), and then one ordered
// pass that counts what lies above it and as many of its equals as are wanted, the first ones.
// evict_move_kernel moves codes, scales and scores, 64 tokens at a time: to other pages all at once, in
// place one workgroup a sequence and head from the front, since a token's new place is never behind its old.
#include "cache.hpp"

namespace gptq {

struct EvictArgs {
    CacheView c;
    Batch q;  // table and lengths; rows and start are not looked at
    float* score;
    int keep, sinks, recent;
    const int32_t* into;  // [seqs, into_width], or NULL: in place
    int into_width;
    int32_t* index;  // [seqs, heads, keep]
    int32_t* length; // [seqs]
    PageDiv div;     // by page / 16
};

constexpr int kSelectThreads = 1024, kSelectBins = 2048;
constexpr int kSelectHeld = 16384, kSelectQuads = kSelectHeld / 4 / kSelectThreads;  // tokens whose keys stay in LDS

// Scores in the order of unsigned numbers: -0 as 0, NaN above all, tokens without a place below all.
__device__ __forceinline__ uint32_t score_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    if (x != x) return ~0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The sum of x over this lane's and lower lanes.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 1; k < 64; k *= 2) {
        const uint32_t y = (uint32_t)__shfl_up((int)x, k);
        if (lane >= k) x += y;
    }
    return x;
}

// One workgroup per sequence and kv head.  Tokens are taken four and four, which lie side by side in their page: one
// look at the table and one vector of scores each, kSelectQuads of them on their way at once.  Bound by latency: 32 x up
// to 8192 tokens of 8 heads take 11 us, lists of 1500 7.
__global__ __launch_bounds__(kSelectThreads) void evict_select_kernel(EvictArgs a) {
    __shared__ u32v4 held[kSelectHeld / 4];  // keys; those of later tokens are made again at each look
    __shared__ __attribute__((aligned(16))) uint32_t bins[kSelectBins];
    __shared__ uint32_t part[2][16];
    __shared__ uint32_t found[3];  // a digit, how many are wanted of those that share it, and how many they are
    const int b = blockIdx.x / a.c.heads, head = blockIdx.x - b * a.c.heads;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t most = (int64_t)a.q.width * a.c.page;
    const int len = (int)min((int64_t)max(a.q.len[b], 0), most), n = min(len, a.keep);
    int32_t* index = a.index + ((int64_t)b * a.c.heads + head) * a.keep;
    if (head == 0 && threadIdx.x == 0) a.length[b] = n;
    for (int j = n + threadIdx.x; j < a.keep; j += kSelectThreads) index[j] = -1;
    if (len == n) {
        for (int j = threadIdx.x; j < n; j += kSelectThreads) index[j] = j;
        return;
    }
    // len > keep >= sinks + recent: tokens from lo to hi - 1 compete for `want` places.
    const int lo = a.sinks, hi = len - a.recent, quads = (len + 3) >> 2;
    uint32_t want = (uint32_t)(a.keep - a.sinks - a.recent);
    const int32_t* table = a.q.table + (int64_t)b * a.q.width;
    // The four scores from token 4 v on (v below `quads`; a page holds whole fours): their place, or -1.
    auto place = [&](int v) -> int64_t {
        const uint32_t blk = (uint32_t)((uint64_t)((uint32_t)v >> 2) * a.div.m >> a.div.shift);
        const int page = table[blk];
        if ((unsigned)page >= (unsigned)a.c.pages) return -1;
        return ((int64_t)page * a.c.heads + head) * a.c.page + (4 * v - (int)blk * a.c.page);
    };
    auto keys_at = [&](int64_t at) {
        u32v4 k = {0u, 0u, 0u, 0u};
        if (at >= 0) {
            const f32v4 x = *(const f32v4*)(a.score + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) k[i] = score_key(x[i]);
        }
        return k;
    };
    {
        int64_t at[kSelectQuads];
#pragma unroll
        for (int i = 0; i < kSelectQuads; ++i) {
            const int v = threadIdx.x + i * kSelectThreads;
            at[i] = v < quads ? place(v) : -1;
        }
#pragma unroll
        for (int i = 0; i < kSelectQuads; ++i) {
            const int v = threadIdx.x + i * kSelectThreads;
            if (v < quads) held[v] = keys_at(at[i]);
        }
    }
    // What a thread put there it reads itself: no barrier in between.
    auto keys = [&](int v) { return v < kSelectHeld / 4 ? held[v] : keys_at(place(v)); };
    // The threshold, as far as it is settled: its bits under the mask `above`.
    uint32_t prefix = 0u, above = 0u;
    int shift = 32;
    bool done = want == 0u;
    if (done) prefix = above = ~0u;  // no place to win: none is above the largest
#pragma unroll 1
    for (int pass = 0; pass < 3 && !done; ++pass) {
        const int bits = pass < 2 ? 11 : 10;
        shift -= bits;
        *(u32v2*)&bins[2 * threadIdx.x] = u32v2{0u, 0u};
        __syncthreads();
        for (int v = threadIdx.x; v < quads; v += kSelectThreads) {
            const u32v4 k = keys(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pos = 4 * v + i;
                if (pos >= lo && pos < hi && ((k[i] ^ prefix) & above) == 0u) atomicAdd(&bins[k[i] >> shift & ((1u << bits) - 1u)], 1u);
            }
        }
        __syncthreads();
        // Two bins a thread, the highest first: counts of all above a thread's own.
        const int top = kSelectBins - 1 - 2 * (int)threadIdx.x;
        const u32v2 two = *(const u32v2*)&bins[top - 1];
        const uint32_t n0 = two[1], n1 = two[0], sum = wave_scan(n0 + n1);
        if (lane == 63) part[0][wave] = sum;
        __syncthreads();
        uint32_t before = sum - n0 - n1;
#pragma unroll
        for (int w = 0; w < 16; ++w) before += w < wave ? part[0][w] : 0u;
        if (before < want && want <= before + n0) {
            found[0] = (uint32_t)top;
            found[1] = want - before;
            found[2] = n0;
        } else if (before + n0 < want && want <= before + n0 + n1) {
            found[0] = (uint32_t)(top - 1);
            found[1] = want - before - n0;
            found[2] = n1;
        }
        __syncthreads();
        prefix |= found[0] << shift;
        above = ~0u << shift;
        want = found[1];
        done = found[2] == want;  // all of them are kept, whatever their lower bits
        // `found` and `part` are written again behind barriers only.
    }
    __syncthreads();
    // Kept in order: those above the threshold, the first `want` of those at it, and the protected.
    uint32_t over = 0u, equal = 0u;  // so far
    int turn = 0;
    for (int v0 = 0; v0 < quads; v0 += kSelectThreads, turn ^= 1) {
        const int v = v0 + threadIdx.x;
        bool gt[4] = {}, eq[4] = {};
        uint32_t mine = 0u;  // counts in halves of 16 bits, up to 4096
        if (v < quads) {
            const u32v4 k = keys(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pos = 4 * v + i;
                const bool fixed = pos < lo || pos >= hi;
                gt[i] = pos < len && (fixed || (k[i] & above) > prefix);
                eq[i] = pos < len && !fixed && (k[i] & above) == prefix;
                mine += (gt[i] ? 1u : 0u) + (eq[i] ? 0x10000u : 0u);
            }
        }
        const uint32_t sum = wave_scan(mine);
        if (lane == 63) part[turn][wave] = sum;
        __syncthreads();
        uint32_t before = sum - mine, all = 0u;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            const uint32_t x = part[turn][w];
            before += w < wave ? x : 0u;
            all += x;
        }
        uint32_t gts = over + (before & 0xffffu), eqs = equal + (before >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (gt[i] || (eq[i] && eqs < want)) index[gts + min(eqs, want)] = 4 * v + i;
            gts += gt[i] ? 1u : 0u;
            eqs += eq[i] ? 1u : 0u;
        }
        over += all & 0xffffu;
        equal += all >> 16;
    }
}

constexpr int kMoveThreads = 256, kMoveTokens = 64;

// Bound by memory's lines of 128 bytes: a kept token's row is 64 of them and lies among others that go, so that twice
// what is needed is read.  2048 of up to 8192 tokens of 32 sequences and 8 heads of 128 channels take 35 us.
// In place a workgroup has a list to itself and waits for memory each 64 tokens: 77 us, and 1024 of 1500 tokens of 8 heads 24
// where 3.4 do to other pages.
template <int G, bool IN_PLACE>
__global__ __launch_bounds__(kMoveThreads) void evict_move_kernel(EvictArgs a) {
    constexpr int PER = 2 * G;                              // 16-byte pieces of a token: G of keys, G of values
    constexpr int TURNS = kMoveTokens * PER / kMoveThreads; // .. a thread
    constexpr int ST = kMoveTokens * G / kMoveThreads > 0 ? kMoveTokens * G / kMoveThreads : 1;  // words of scales a thread
    __shared__ int64_t from[kMoveTokens], to[kMoveTokens];
    const int bh = blockIdx.x, b = bh / a.c.heads, head = bh - b * a.c.heads;
    const int n = a.length[b];
    Batch into = a.q;
    if constexpr (!IN_PLACE) {
        into.table = a.into;
        into.width = a.into_width;
    }
    const int32_t* index = a.index + (int64_t)bh * a.keep;
    const int step = IN_PLACE ? 1 : (int)gridDim.y;
    for (int64_t tile = IN_PLACE ? 0 : blockIdx.y; tile * kMoveTokens < n; tile += step) {
        const int j0 = (int)(tile * kMoveTokens);
        if (threadIdx.x < kMoveTokens) {
            const int j = j0 + threadIdx.x;
            int64_t f = -1, t = -1;
            if (j < n) {
                const int old = index[j];
                f = cache_row(a.c, a.q, b, old, head);
                t = cache_row(a.c, into, b, j, head);
                if (IN_PLACE && old == j) t = -1;  // stays
            }
            from[threadIdx.x] = f;
            to[threadIdx.x] = t;
        }
        __syncthreads();
        // A token without a place has codes and scales of 0.
        u32v4 v[TURNS];
#pragma unroll
        for (int k = 0; k < TURNS; ++k) {
            const int u = k * kMoveThreads + threadIdx.x, tok = u / PER, piece = u % PER;
            const int64_t f = from[tok];
            v[k] = u32v4{0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
            if (f >= 0 && to[tok] >= 0) v[k] = *(const u32v4*)((piece < G ? a.c.k : a.c.v) + f * (16 * G) + (piece % G) * 16);
        }
        // Scales: G / 2 words of keys and as many of values a token; scores one.
        uint32_t sc[ST];
#pragma unroll
        for (int k = 0; k < ST; ++k) {
            const int u = k * kMoveThreads + threadIdx.x, tok = u / G, word = u % G;
            sc[k] = 0u;
            if (u < kMoveTokens * G) {
                const int64_t f = from[tok];
                if (f >= 0 && to[tok] >= 0) sc[k] = ((const uint32_t*)((word < G / 2 ? a.c.ks : a.c.vs) + f * G))[word % (G / 2)];
            }
        }
        float score = 0.0f;
        if (threadIdx.x < kMoveTokens && from[threadIdx.x] >= 0 && to[threadIdx.x] >= 0) score = a.score[from[threadIdx.x]];
        if constexpr (IN_PLACE) {
            // Every read of the tile has returned before any of its places is written; what is read later
            // lies behind them.
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < TURNS; ++k) {
            const int u = k * kMoveThreads + threadIdx.x, tok = u / PER, piece = u % PER;
            const int64_t t = to[tok];
            if (t >= 0) *(u32v4*)((piece < G ? a.c.k : a.c.v) + t * (16 * G) + (piece % G) * 16) = v[k];
        }
#pragma unroll
        for (int k = 0; k < ST; ++k) {
            const int u = k * kMoveThreads + threadIdx.x, tok = u / G, word = u % G;
            if (u < kMoveTokens * G) {
                const int64_t t = to[tok];
                if (t >= 0) ((uint32_t*)((word < G / 2 ? a.c.ks : a.c.vs) + t * G))[word % (G / 2)] = sc[k];
            }
        }
        if (threadIdx.x < kMoveTokens && to[threadIdx.x] >= 0) a.score[to[threadIdx.x]] = score;
        __syncthreads();
    }
}

typedef void (*MoveKernel)(EvictArgs);
template <bool IN_PLACE>
static MoveKernel move_pick(int dim) {
    return dim == 64 ? evict_move_kernel<2, IN_PLACE> : dim == 128 ? evict_move_kernel<4, IN_PLACE> : evict_move_kernel<8, IN_PLACE>;
}

}  // namespace gptq

using namespace gptq;

extern "C" int gptq_cache_evict(const gptq_cache* cache, const gptq_batch* batch, float* score, int32_t keep, int32_t sinks,
                                int32_t recent, const int32_t* into, int32_t into_width, int32_t* length, int32_t* index,
                                void* stream) {
    if (!cache_ok(cache) || !batch || !table_ok(cache, batch)) return GPTQ_EINVAL;
    gptq_batch whole = *batch;  // whole sequences: no rows of a call
    whole.start = nullptr;
    whole.rows = whole.seqs;
    if (!batch_ok(&whole)) return GPTQ_EINVAL;
    if (keep < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > keep || keep > (1 << 30)) return GPTQ_EINVAL;
    if (!score || !length || !index || !al16(score) || (((uintptr_t)length | (uintptr_t)index | (uintptr_t)into) & 3u)) return GPTQ_EINVAL;
    if (into && (into_width < 1 || into_width > (1 << 24) || (int64_t)into_width * cache->page > (1 << 30))) return GPTQ_EINVAL;
    const int64_t lists = whole.seqs * (int64_t)cache->heads;
    // A launch has fewer than 2^32 threads.
    if (lists * kSelectThreads > ((int64_t)1 << 32) - 1 || lists > ((int64_t)1 << 40) / keep) return GPTQ_EINVAL;
    const int64_t tokens = cache->pages * cache->page * cache->heads;
    auto set = [](const void* p, int64_t bytes) { return RowSet{p, bytes, p ? 1 : 0, bytes}; };
    const RowSet s = set(score, 4 * tokens), l = set(length, 4 * (int64_t)whole.seqs), x = set(index, 4 * lists * keep);
    const RowSet in[] = {set(whole.table, 4 * (int64_t)whole.seqs * whole.width), set(whole.len, 4 * (int64_t)whole.seqs),
                         set(into, 4 * (int64_t)whole.seqs * into_width)};
    for (const RowSet& o : {s, l, x}) {
        if (meets_cache(o, cache)) return GPTQ_EINVAL;
        for (const RowSet& i : in)
            if (rows_meet(o, i)) return GPTQ_EINVAL;
    }
    if (rows_meet(s, l) || rows_meet(s, x) || rows_meet(l, x)) return GPTQ_EINVAL;
    CheckScope check;
    check_cache(cache, &whole);
    check_buffer(score, sizeof(float) * (size_t)tokens, "score");
    check_buffer(length, 4 * (size_t)whole.seqs, "length");
    check_buffer(index, 4 * (size_t)(lists * keep), "index");
    if (into) check_buffer(into, 4 * (size_t)whole.seqs * (size_t)into_width, "into");
    hipStream_t st = (hipStream_t)stream;
    const EvictArgs a{cache_view(cache), batch_view(&whole), score, keep, sinks, recent, into, into_width, index, length, page_div(cache->page)};
    {
        ProfScope ps(FAM_CACHE, st, 0.0, 0.0);
        GPTQ_LAUNCH(st, "evict_select", (evict_select_kernel<<<(unsigned)lists, kSelectThreads, 0, st>>>(a)), batch_span(&whole, 0),
                    batch_span(&whole, 1), rd(score, tokens, 1, tokens), wr(index, keep, lists, keep), wr(length, whole.seqs, 1, whole.seqs));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    int64_t tiles = ((int64_t)keep + kMoveTokens - 1) / kMoveTokens;
    if (tiles > 32768) tiles = 32768;
    const MoveKernel k = into ? move_pick<false>(cache->dim) : move_pick<true>(cache->dim);
    {
        ProfScope ps(FAM_CACHE, st, 0.0, 0.0);
        GPTQ_LAUNCH(st, "evict_move", (k<<<dim3((unsigned)lists, into ? (unsigned)tiles : 1u), kMoveThreads, 0, st>>>(a)),
                    batch_span(&whole, 0), rd(index, keep, lists, keep), rd(length, whole.seqs, 1, whole.seqs),
                    rd(into ? into : whole.table, into ? into_width : whole.width, whole.seqs, into ? into_width : whole.width),
                    plane(cache->k, cache, cache->dim / 2, true), plane(cache->v, cache, cache->dim / 2, true),
                    plane(cache->k_scale, cache, cache->dim / 16, true), plane(cache->v_scale, cache, cache->dim / 16, true),
                    wr(score, tokens, 1, tokens));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}
