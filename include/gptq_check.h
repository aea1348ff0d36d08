/*
 * gptq_check.h -- schedule checking of libgptq_mi355x (a dry run for tests; no GPU needed).
 *
 * With check mode on, gptq_fold, gptq_ladder and gptq_sweep run their host-side schedule
 * without any HIP call: no kernel is launched, no stream or event is touched, device pointers
 * are never dereferenced (any distinct addresses of the right sizes will do) and the fold's
 * pivot flag reads as clear.  Every launch instead records the 2-D spans of memory it reads and
 * writes, and every event record / stream wait / host synchronisation is simulated with
 * vector clocks over the streams.  The call then returns GPTQ_ECHECK if
 *   - a span leaves every buffer the call was given (inputs, outputs, workspace), or
 *   - two launches on different streams touch overlapping memory, one of them writing, and
 *     neither is ordered before the other;
 * otherwise its usual status.  gptq_check_message() describes the first failure of the last
 * checked call on any thread ("" when it passed).  The mode is process-wide; calls made while
 * it is on must not expect results.
 */
#ifndef GPTQ_MI355X_CHECK_H
#define GPTQ_MI355X_CHECK_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

void gptq_check_mode(int on);
const char* gptq_check_message(void);
/* The checker on a fixed hand-made schedule: 0 clean (GPTQ_OK), 1 an unordered overlapping
 * write (GPTQ_ECHECK), 2 the same ordered by an event (GPTQ_OK), 3 a read past the end of
 * its buffer (GPTQ_ECHECK). */
int gptq_check_selftest(int which);
/* The tile GEMM's map from workgroup to output tile, on the host: GPTQ_OK when the workgroups
 * of one launch over an M x N product (lower != 0: the lower tiles of an M x M product, N
 * ignored) cover every 128 x 128 tile exactly once, for each group of a batched launch (grid
 * z = 0 .. 15); GPTQ_ECHECK otherwise; GPTQ_EINVAL for sizes outside 1 .. 2^20. */
int gptq_check_tile_order(int64_t M, int64_t N, int lower);
/* Where the cache kernels keep a position, on the host: the index of the (page, head, token) row
 * of position `pos` of sequence `seq` (table: a HOST array, [seqs, width]), or -1 where the cache
 * has no such place. */
int64_t gptq_check_cache_row(int64_t pages, int32_t page, int32_t heads, int32_t width,
                             const int32_t* table, int32_t seq, int64_t pos, int32_t head);
/* How gptq_linear lays a size out, on the host (dtype as in that call): plan[0] the kernel (1
 * linear_codes_kernel, 2 linear_tile_kernel, 3 dense_kernel on decoded weights), plan[1] the pieces of K
 * (3: of each cut tile), plan[2] and plan[3] the tiles taken whole and the tiles cut (3 only, else 0).
 * GPTQ_EINVAL for sizes that the call refuses. */
int gptq_check_linear_plan(int dtype, int64_t t, int64_t rows, int64_t n, int64_t* plan);
/* The attention's cut of a sequence into blocks of tokens, on the host: GPTQ_OK when, for `rows` rows
 * at the end of `len` tokens (`held` of which the table can hold), tiles of `rows_tile` rows and
 * blocks of `block` tokens, every key that a row sees is in
 * exactly one block of the row's tile, and blocks taken without a mask hold no key that one of the
 * tile's rows does not see; GPTQ_ECHECK otherwise. */
int gptq_check_attention_blocks(int32_t len, int32_t rows, int32_t group, int64_t held, int32_t window,
                                int32_t sinks, int32_t splits, int32_t rows_tile, int32_t block);

#ifdef __cplusplus
}
#endif
#endif
