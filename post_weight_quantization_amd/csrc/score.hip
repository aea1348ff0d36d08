// score.hip -- the attention that cached tokens have received, on gfx950.
//
//   score[t] = old[t] + sum over the call's rows and a kv head's query heads of e^(scale q k_t - lse),
// lse the row's own (gptq_cache_attention's): the softmax weights of the whole call, added up by token.
//
// Tokens own the work: a wave holds the keys of 16 TT tokens of one kv head as matrix operands (c s, exact in
// bf16) and walks over the query rows that see them, 16 at a time.  Scores come as in the attention's tile
// kernel, tokens in D's rows and queries in its columns; a lane adds its own queries' weights, the sixteen
// columns are added at the end.  So no sum is shared by waves, nothing is joined, and results do not depend
// on timing.
#include <math.h>

#include "attention.hpp"

namespace gptq {

struct ScoreArgs {
    AttnArgs a;        // lse is read here
    const float* old;  // [pages, heads, page]
    float* out;        // the same places; may be old itself
    int tiles;         // workgroups along a sequence; each takes every tiles-th piece of it
};

constexpr int kScoreWaves = 4;
template <int G>
constexpr int kScoreTiles = G == 8 ? 2 : 4;  // 16-token tiles of a wave: keys in 64 registers (dim 64: 32)

// x summed over the 16 lanes of each row of the wave, in every lane.
__device__ __forceinline__ float row_sum(float x) {
#define GPTQ_ADD_ROTATED(N) x += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x120 + N, 0xf, 0xf, false))
    GPTQ_ADD_ROTATED(8);
    GPTQ_ADD_ROTATED(4);
    GPTQ_ADD_ROTATED(2);
    GPTQ_ADD_ROTATED(1);
#undef GPTQ_ADD_ROTATED
    return x;
}

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

template <int DT, int G>
__global__ __launch_bounds__(kScoreWaves * 64) void score_kernel(ScoreArgs s) {
    constexpr int NT = kTerms<DT>, TT = kScoreTiles<G>, TOK = 16 * TT;
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
    const int len = max(a.q.len[b], 0), pos0 = len - R, end = (int)min((int64_t)len, held);
    const int32_t* table = a.q.table + (int64_t)b * a.q.width;
    for (int64_t at = ((int64_t)first * kScoreWaves + wave) * TOK; at < end; at += (int64_t)s.tiles * kScoreWaves * TOK) {
        const int tok0 = (int)at;
        u32v4 key[TT][G];
        int64_t place[TT];
        bool there[TT];
#pragma unroll
        for (int u = 0; u < TT; ++u) {
            place[u] = find_page(a, table, head, tok0 + 16 * u, there[u]);
            uint32_t w[G];
            load_key_words<G>(a.c.k + (place[u] + c) * (16 * G) + h * (4 * G), w);
            const uint32_t* sp = (const uint32_t*)(a.c.ks + (place[u] + c) * G);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const uint32_t x = sp[i >> 1];
                const float z = __uint_as_float((i & 1) ? x & 0xffff0000u : x << 16), z8 = -8.0f * z;
                const uint32_t even = nibble_bytes(w[i], false), odd = nibble_bytes(w[i], true);
                key[u][i] = u32v4{decode_pair<0, 2>(even, z, z8, z, z8), decode_pair<0, 2>(odd, z, z8, z, z8),
                                  decode_pair<1, 3>(even, z, z8, z, z8), decode_pair<1, 3>(odd, z, z8, z, z8)};
            }
        }
        float sum[TT][4];
#pragma unroll
        for (int u = 0; u < TT; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[u][r] = 0.0f;
        int x0, x1;
        score_rows(tok0, tok0 + TOK, pos0, R, a.group, a.window, a.sinks, x0, x1);
        for (int x = x0; x < x1; x += 16) {
            const int xq = min(x + c, x1 - 1), qi = xq / a.group, qh = head * a.group + (xq - qi * a.group);
            const int64_t row = r0 + qi;
            const float lse = a.lse[row * a.qheads + qh] * 1.4426950408889634f;
            f32v4 d[TT];
#pragma unroll
            for (int u = 0; u < TT; ++u) d[u] = f32v4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < G; ++i) {
                u32v4 q[NT];
                load_terms<DT, false>(a.Q, row * a.ldq + (int64_t)qh * a.ldqh + 32 * i + 8 * h, q);
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    q[k] ^= a.flip;
#pragma unroll
                    for (int u = 0; u < TT; ++u) d[u] = mfma16(key[u][i], q[k], d[u]);
                }
            }
            // A row that sees nothing has lse = -inf and pays nothing.
            const bool pays = x + c < x1 && lse != -INFINITY;
            const int qpos = pos0 + qi, low = window_low(qpos, a.window);
#pragma unroll
            for (int u = 0; u < TT; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(d[u][r], a.scale2, -lse));
                    const bool seen = pays & key_seen(tok0 + 16 * u + 4 * h + r, qpos, low, a.sinks);
                    sum[u][r] += seen ? p : 0.0f;
                }
        }
#pragma unroll
        for (int u = 0; u < TT; ++u) {
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[u][r] = row_sum(sum[u][r]);
            // Lane r of each quarter writes token r of its four.
            const int tok = tok0 + 16 * u + 4 * h + c;
            const float mine = c == 0 ? sum[u][0] : c == 1 ? sum[u][1] : c == 2 ? sum[u][2] : sum[u][3];
            if (there[u] && c < 4 && tok < end) {
                const int64_t to = place[u] + 4 * h + c;
                s.out[to] = tok < pos0 ? s.old[to] + mine : mine;
            }
        }
    }
}

typedef void (*ScoreKernel)(ScoreArgs);
template <int DT>
static ScoreKernel score_pick(int dim) {
    return dim == 64 ? score_kernel<DT, 2> : dim == 128 ? score_kernel<DT, 4> : score_kernel<DT, 8>;
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
    const int64_t piece = kScoreWaves * 16 * (cache->dim == 256 ? 2 : 4);
    int64_t tiles = ((int64_t)batch->width * cache->page + piece - 1) / piece;
    // Workgroups past a grid's size, or many rounds of them: each takes several pieces of its sequence.
    const int64_t most = ((int64_t)1 << 20) / ((int64_t)cache->heads * (batch->seqs < 16 ? batch->seqs : 16)) + 1;
    if (tiles > most) tiles = most;
    s.tiles = (int)tiles;
    const ScoreKernel k = dtype == GPTQ_F32 ? score_pick<GPTQ_F32>(cache->dim) : dtype == GPTQ_BF16 ? score_pick<GPTQ_BF16>(cache->dim) : score_pick<GPTQ_F16>(cache->dim);
    const int64_t qw = (q_heads - 1) * ldqh + cache->dim, seqs = batch->seqs;
    const Span none = rd(score, tokens, 0, tokens);
    {
        ProfScope ps(FAM_ATTENTION, st, 0.0, 0.0);
        GPTQ_LAUNCH(st, "cache_score",
                    (k<<<dim3((unsigned)(cache->heads * tiles), (unsigned)(seqs < kGridTiles ? seqs : kGridTiles),
                              (unsigned)((seqs + kGridTiles - 1) / kGridTiles)), kScoreWaves * 64, 0, st>>>(s)),
                    batch->rows ? rd(Q, ldq, batch->rows, qw, es) : none, batch->rows ? rd(lse, items, 1, items) : none,
                    batch_span(batch, 0), batch_span(batch, 1), batch_span(batch, 2), plane(cache->k, cache, cache->dim / 2, false),
                    plane(cache->k_scale, cache, cache->dim / 16, false), rd(score, tokens, 1, tokens), wr(out, tokens, 1, tokens));
    }
    if (launch_status() != GPTQ_OK) return GPTQ_EHIP;
    return check.finish();
}
