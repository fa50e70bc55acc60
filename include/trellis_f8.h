/*
 * trellis_f8.h -- the parts of a model step that stay in a checkpoint's block-scaled FP8, next to
 * the trellis-coded products, on AMD Instinct MI355X (gfx950): the norm in front of a product,
 * the gated activation, and products against E4M3 matrices, one or one per expert.
 *
 * Format.  A row of n channels is stored as n E4M3 codes (OCP: bias 7, no infinities, largest
 * finite 448) and ceil(n / 128) f32 scales: channel c stands for code(c) * scale(c / 128).  A
 * matrix [out][in] has one scale per 128 x 128 block, [ceil(out / 128)][ceil(in / 128)].
 * Quantising a block: a = max |v|, scale = a / 448, code = v / scale to the nearest E4M3 value,
 * ties to even.  A block whose scale is below the smallest normal f32 (a block of zeros, too) is
 * stored as scale 0 and codes 0; one with an infinity or NaN as scale NaN and codes 0: it stands
 * for NaN.  Values are formed in f32 before they are quantised or rounded: one above its largest
 * number (products of bf16's largest) is an infinity.
 *
 * Conventions as in trellis.h: device pointers unless stated otherwise, `stream` a hipStream_t
 * as void*, calls only enqueue, nothing is allocated, validation on the host before anything is
 * enqueued.  Strides are in elements.  The products take a caller-owned zero-filled workspace
 * that every entry point of the library can share on one stream.  What only the device can see
 * (offsets, row lists) is checked in the kernels: a bad value is never used as an address, and
 * bit 1 of the workspace's error word is set.
 */
#ifndef TRELLIS_F8_H_
#define TRELLIS_F8_H_

#include <stddef.h>
#include <stdint.h>

#include "trellis.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of 16-bit inputs and outputs. */
enum { TRELLIS_F8_F16 = 0, TRELLIS_F8_BF16 = 1 };

/* E4M3 matrices (passed by HOST pointer): w [n_experts][out][in], scale f32 [n_experts]
 * [ceil(out / 128)][ceil(in / 128)].  in a multiple of 16 (a last block may be partial), w
 * 16-byte aligned.  n_experts = 1 for one matrix. */
typedef struct {
  const uint8_t *w;
  const float *scale;
  int32_t n_experts;
  int32_t in_features;
  int32_t out_features;
} trellis_f8_linear;

/* Root-mean-square norm of rows, with the residual's addition and an E4M3 result:
 *   h = x + residual (f32; x alone if residual is NULL),
 *   v = h * gamma / sqrt(mean(h^2) + eps)          (gamma NULL: ones)
 *   q, scale = v quantised per block of 128; y = v rounded to `dtype`; h_out = h rounded.
 * x       : [rows][n] of `dtype` at row stride x_row (a multiple of 8); residual [rows][n], dense.
 * gamma   : [n] of `dtype`.
 * q, scale: E4M3 out [rows][n] and f32 out [rows][ceil(n / 128)]; both or neither (NULL).
 * y       : out [rows][n] for products that take 16 bits, or NULL; one of q and y is given.
 * h_out   : out [rows][n], the next residual, or NULL; may be x (if dense) or residual.
 * n a multiple of 16, at most 32768; rows below 2^22; eps at least the smallest normal f32 and finite; arrays
 * 16-byte aligned.  Outputs may not overlap each other, nor inputs except as said.  One launch. */
int trellis_f8_norm(int dtype, const void *x, int64_t x_row, const void *residual, const void *gamma, int rows, int n,
                    float eps, void *h_out, uint8_t *q, float *scale, void *y, void *stream);

/* Gated activation: v = silu(g) * u, silu(z) = z / (1 + e^-z), of rows that hold g in their
 * first n channels and u in the next n; q, scale, y as for trellis_f8_norm.
 * x: [rows][2n] of `dtype` at row stride x_row (a multiple of 8, at least 2n).  n a multiple of
 * 16; arrays 16-byte aligned; no output may overlap x.  One launch. */
int trellis_f8_silu_mul(int dtype, const void *x, int64_t x_row, int rows, int n, uint8_t *q, float *scale, void *y,
                        void *stream);

/* Bytes of workspace trellis_f8_gemm needs for M rows, trellis_f8_moe_gemm for `rows` rows
 * (0 for invalid arguments).  Host pointer L. */
size_t trellis_f8_gemm_workspace_bytes(const trellis_f8_linear *L, int M);
size_t trellis_f8_moe_gemm_workspace_bytes(const trellis_f8_linear *L, int rows);

/* y[m][o] = sum_b s[m][b] sw[o / 128][b] sum_{c in block b} q[m][c] w[o][c], summed in f32 but
 * for the matrix instruction's sums of eight neighbouring channels' products, whose terms are held
 * in steps of 2^-13 of the largest one's power of two.
 * s sw is formed in f32: a product below its smallest normal number is held in steps of 2^-149, which
 * moves a result by less than 2^-125 for each block; one above its largest is no part of the result
 * (s and sw meet the block's sum one after the other there).
 * L    : HOST pointer, n_experts = 1.
 * q    : E4M3 [M][in] at row stride q_row (a multiple of 16), 16-byte aligned; s: f32 [M]
 *        [ceil(in / 128)] at row stride s_row.
 * y    : out [M][out] of `dtype` at row stride y_row (at least out); must not overlap an input.
 * M >= 0 (0 is a no-op), any out_features; ws: >= trellis_f8_gemm_workspace_bytes().
 * The result does not depend on timing: sums that several workgroups share are joined in a fixed
 * order.  One launch, two where the blocks of few tiles are shared among workgroups. */
int trellis_f8_gemm(const trellis_f8_linear *L, const uint8_t *q, int64_t q_row, const float *s, int64_t s_row, int M,
                    int dtype, void *y, int64_t y_row, void *ws, size_t ws_bytes, void *stream);

/* The same for rows sorted by expert: row r in [offsets[e], offsets[e+1]) is multiplied by
 * matrix e.
 * offsets: DEVICE int32 [n_experts + 1] from 0, ascending, its last at most `rows`; where it is
 *          not, the call ends there (bit 1).  Rows of y from its last entry on are left alone.
 * order  : NULL: row r is row r of q; or DEVICE int32 [rows]: row r is row order[r] / per of q
 *          (trellis_moe_sort's list with per = experts a token: nothing is gathered first).  A
 *          quotient outside [0, n_q) gives a zero row (bit 1).
 * n_q    : rows of q and s (>= rows if order is NULL).   rows: of y. */
int trellis_f8_moe_gemm(const trellis_f8_linear *L, const uint8_t *q, int64_t q_row, const float *s, int64_t s_row,
                        int n_q, const int32_t *offsets, const int32_t *order, int per, int rows, int dtype, void *y,
                        int64_t y_row, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TRELLIS_F8_H_ */
