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
};

constexpr int kSelectThreads = 1024, kSelectBins = 2048, kSelectHeld = 8192;

// Scores in the order of unsigned numbers: -0 as 0, NaN above all, tokens without a place below all.
__device__ __forceinline__ uint32_t score_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    if (x != x) return ~0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ __launch_bounds__(kSelectThreads) void evict_select_kernel(EvictArgs a) {
    __shared__ uint32_t held[kSelectHeld];  // keys of the first tokens between; the others are read again
    __shared__ uint32_t bins[kSelectBins];
    __shared__ uint32_t part[2][16];
    __shared__ uint32_t found[2];  // a digit and how many are wanted of those that share it
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
    const int lo = a.sinks, hi = len - a.recent;
    uint32_t want = (uint32_t)(a.keep - a.sinks - a.recent);
    auto look = [&](int pos) -> uint32_t {
        const int64_t at = cache_row(a.c, a.q, b, pos, head);
        return at < 0 ? 0u : score_key(a.score[at]);
    };
    for (int i = threadIdx.x; i < min(hi - lo, kSelectHeld); i += kSelectThreads) held[i] = look(lo + i);
    auto key = [&](int pos) { return pos - lo < kSelectHeld ? held[pos - lo] : look(pos); };
    uint32_t prefix = 0u;
    int shift = 32;
    // With no place to win, all keys stay below the threshold: none is above the largest.
    if (want == 0u) prefix = ~0u;
#pragma unroll 1
    for (int pass = 0; pass < 3 && want; ++pass) {
        const int bits = pass < 2 ? 11 : 10;
        const uint32_t above = pass ? ~0u << shift : 0u;  // bits that are settled
        shift -= bits;
        for (int i = threadIdx.x; i < kSelectBins; i += kSelectThreads) bins[i] = 0u;
        __syncthreads();
        for (int pos = lo + threadIdx.x; pos < hi; pos += kSelectThreads) {
            const uint32_t k = key(pos);
            if (((k ^ prefix) & above) == 0u) atomicAdd(&bins[k >> shift & ((1u << bits) - 1u)], 1u);
        }
        __syncthreads();
        // Two bins a thread, the highest first: counts of all above a thread's own.
        const int top = kSelectBins - 1 - 2 * (int)threadIdx.x;
        const uint32_t n0 = bins[top], n1 = bins[top - 1];
        uint32_t sum = n0 + n1;
#pragma unroll
        for (int k = 1; k < 64; k *= 2) {
            const uint32_t y = (uint32_t)__shfl_up((int)sum, k);
            if (lane >= k) sum += y;
        }
        if (lane == 63) part[0][wave] = sum;
        __syncthreads();
        uint32_t before = sum - n0 - n1;
        for (int w = 0; w < wave; ++w) before += part[0][w];
        if (before < want && want <= before + n0) {
            found[0] = (uint32_t)top;
            found[1] = want - before;
        } else if (before + n0 < want && want <= before + n0 + n1) {
            found[0] = (uint32_t)(top - 1);
            found[1] = want - before - n0;
        }
        __syncthreads();
        prefix |= found[0] << shift;
        want = found[1];
        // `found` and `part` are written again behind barriers only.
    }
    __syncthreads();
    // Kept in order: those above the threshold, the first `want` of those at it, and the protected.
    uint32_t over = 0u, equal = 0u;  // so far
    int turn = 0;
    for (int p0 = 0; p0 < len; p0 += kSelectThreads, turn ^= 1) {
        const int pos = p0 + threadIdx.x;
        bool gt = false, eq = false;
        if (pos < len) {
            if (pos < lo || pos >= hi) {
                gt = true;
            } else {
                const uint32_t k = key(pos);
                gt = k > prefix;
                eq = k == prefix;
            }
        }
        const unsigned long long g = __ballot(gt), e = __ballot(eq), below = (1ull << lane) - 1ull;
        if (lane == 0) part[turn][wave] = (uint32_t)__popcll(g) | (uint32_t)__popcll(e) << 16;
        __syncthreads();
        uint32_t before = 0u, all = 0u;  // of this turn: counts in halves of 16 bits, up to 1024
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            const uint32_t x = part[turn][w];
            if (w < wave) before += x;
            all += x;
        }
        const uint32_t gts = over + (before & 0xffffu) + (uint32_t)__popcll(g & below);
        const uint32_t eqs = equal + (before >> 16) + (uint32_t)__popcll(e & below);
        if (gt || (eq && eqs < want)) index[gts + min(eqs, want)] = pos;
        over += all & 0xffffu;
        equal += all >> 16;
    }
}

constexpr int kMoveThreads = 256, kMoveTokens = 64;

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
    if (!score || !length || !index || (((uintptr_t)score | (uintptr_t)length | (uintptr_t)index | (uintptr_t)into) & 3u)) return GPTQ_EINVAL;
    if (into && (into_width < 1 || into_width > (1 << 24) || (int64_t)into_width * cache->page > (1 << 30))) return GPTQ_EINVAL;
    const int64_t lists = whole.seqs * (int64_t)cache->heads;
    if (lists > ((int64_t)1 << 31) - 1 || lists > ((int64_t)1 << 40) / keep) return GPTQ_EINVAL;
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
    const EvictArgs a{cache_view(cache), batch_view(&whole), score, keep, sinks, recent, into, into_width, index, length};
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
