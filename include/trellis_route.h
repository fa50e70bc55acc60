/*
 * trellis_route.h -- tokens of a batch sorted by their routed experts, and back with the router's
 * weights, on AMD Instinct MI355X (gfx950): what stands around the experts' products when there
 * is more than one token (trellis_moe_mlp is one token's), forwards and backwards.
 *
 * An ENTRY is one (token, choice) pair, entry t * top + j for choice j of token t.  Sorted by
 * expert, ties by entry, the entries whose expert is here take the POSITIONS 0, 1, ...; position
 * p is row p of the arrays that the experts' products read and write.
 *
 * Conventions as in trellis.h: device pointers, `stream` a hipStream_t as void*, calls only
 * enqueue, nothing is allocated, validation on the host before anything is enqueued, a
 * caller-owned zero-filled workspace that every entry point of the library can share on one
 * stream.  Lists are checked in the kernels: a bad value is never used as an address, what it
 * stands for is skipped, and bit 1 of the workspace's error word is set.
 */
#ifndef TRELLIS_ROUTE_H_
#define TRELLIS_ROUTE_H_

#include <stddef.h>
#include <stdint.h>

#include "trellis.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes: of the sort (0 for invalid sizes) ... */
size_t trellis_moe_sort_workspace_bytes(int tokens, int top, int n_experts);
/* ... of gather, combine and combine_grad (any sizes). */
size_t trellis_moe_rows_workspace_bytes(void);

/* Sort a routing.
 * ids    : int32 [tokens][top]; an id of -1 is an expert that is not here; other ids outside
 *          [0, n_experts) are taken as -1 (bit 1).  A token may name an expert twice.
 * offsets: int32 out [n_experts + 1]: expert e has the positions offsets[e] .. offsets[e+1]-1.
 * order  : int32 out [tokens * top]: the entry at each position; -1 behind the last position.
 * inverse: int32 out [tokens][top]: each entry's position, -1 where its expert is not here.
 * 1 <= n_experts <= 2048, 1 <= top <= 1024, tokens * top <= 2^24.  No output may overlap ids.
 * One launch, three for more than 65536 entries. */
int trellis_moe_sort(const int32_t *ids, int tokens, int top, int n_experts, int32_t *offsets, int32_t *order,
                     int32_t *inverse, void *ws, size_t ws_bytes, void *stream);

/* Tokens' rows brought into the experts' order: row p of out = row order[p] / per of x; rows
 * whose entry is -1 are left alone.  Rows of any type: row_bytes bytes, a multiple of 4, x at a
 * stride of x_row_bytes (a multiple of 4), out dense; pointers 4-byte aligned (16 where
 * row_bytes and stride are multiples of 16 is faster).  out must not overlap x.  One launch.
 * Its gradient is trellis_moe_combine without weights. */
int trellis_moe_gather(const void *x, int64_t x_row_bytes, int tokens, int64_t row_bytes, const int32_t *order, int rows,
                       int per, void *out, void *ws, size_t ws_bytes, void *stream);

/* Back, with weights: out[t] = add[t] + sum_j weights[t][j] * y[inverse[t][j]] over the entries
 * that have a position, in the order of j, summed in f32.
 * y: [rows][n] of dtype (0 fp16, 1 bf16); inverse int32 [tokens][top]; weights f32 [tokens][top]
 * or NULL (ones); add: [tokens][n] of dtype or NULL (zeros).  out: [tokens][n], may be add, must
 * not overlap another input.  n a multiple of 8; arrays dense, y, add and out 16-byte aligned.
 * One launch. */
int trellis_moe_combine(int dtype, const void *y, int rows, int n, const int32_t *inverse, const float *weights,
                        int tokens, int top, const void *add, void *out, void *ws, size_t ws_bytes, void *stream);

/* The gradient of trellis_moe_combine for the gradient d_out [tokens][n] of its result:
 *   d_y[inverse[t][j]] = weights[t][j] * d_out[t]       (rows that no entry names are left alone)
 *   d_weights[t][j] = sum_c d_out[t][c] * y[inverse[t][j]][c], 0 for entries without a position.
 * (That of add is d_out.)  weights NULL: ones.  d_weights f32 [tokens][top] or NULL; y is read
 * for it alone and may be NULL without it.  d_y: [rows][n]; may be y, must not overlap another
 * input.  The positions in inverse are distinct.  One launch. */
int trellis_moe_combine_grad(int dtype, const void *d_out, const void *y, int rows, int n, const int32_t *inverse,
                             const float *weights, int tokens, int top, void *d_y, float *d_weights, void *ws,
                             size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TRELLIS_ROUTE_H_ */
