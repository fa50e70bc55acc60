/*
 * trellis_kv4.h -- a paged key/value cache held in 4 bits, and what a serving loop does with
 * it, on AMD Instinct MI355X (gfx950): append, read back, attention, and the page operations
 * (reserve, fork, compact, free).  It stands between the products of trellis.h: a decode step
 * is the qkv product (trellis_gemv_list), trellis_kv4_append, trellis_kv4_attn and the output
 * product.
 *
 * Format.  A head's vector is split into blocks of 128 (head_dim / 128 = NB of them).  A block
 * x is rotated with the library's Hadamard, r = H_128 x / sqrt(128), and stored as one bf16
 * scale s = bf16(max|r| * (1/6)) and 128 E2M1 codes, the nearest (ties to even) of r * (1/s):
 * magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 in the low three bits, the sign in bit 3.  The rotation
 * spreads a channel that stands out over its block, so one scale per block serves; it is
 * orthogonal, so scores of rotated queries against rotated keys are the scores.  4.125 bits
 * per value.
 *   pool  : [n_layers][n_pages][n_kv_heads][chunk], chunk = 132 * NB * T bytes for T = page_size:
 *           key codes [NB][T][64] | value codes [NB][T][64] | key scales [NB][T] bf16 | value
 *           scales [NB][T] bf16; element d of a block is nibble d % 2 (0 = low) of byte d / 2.
 *   A block with an infinity or NaN (or whose rotation overflows fp32) has scale NaN and codes
 *   0: it stands for NaN.  A block whose scale is below the smallest normal bf16 is stored as 0.
 *
 * Sequences.  A sequence is a slot: a row of the page table and a length.  Token p of slot r is
 * row p % T of page table[r * max_pages + p / T].  ref[page] counts the slots that hold a page
 * (0 = free).  All of it is device memory that the caller owns and the calls update, so a
 * serving loop can be captured in a graph.
 *
 * Conventions as in trellis.h: device pointers unless stated otherwise, `stream` a hipStream_t
 * as void*, calls only enqueue, nothing is allocated, validation on the host before anything is
 * enqueued, a caller-owned zero-filled workspace that every entry point of the library can
 * share on one stream.  What only the device can see (page numbers, slots, lengths) is checked
 * in the kernels: a bad value is never used as an address; the row concerned is skipped (append,
 * a compaction's row) or zero (read, attn) and bit 4 of the workspace's error word is set.  A cu that
 * does not start at 0, descends or passes the rows ends a call of attn there: what follows is zero.  The
 * page operations refuse a call with a bad slot or length as a whole (bit 4), and one that
 * needs more free pages than there are (bit 8): nothing is changed then.
 */
#ifndef TRELLIS_KV4_H_
#define TRELLIS_KV4_H_

#include <stddef.h>
#include <stdint.h>

#include "trellis.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of keys, values, queries and outputs. */
enum { TRELLIS_KV4_F16 = 0, TRELLIS_KV4_BF16 = 1 };

/* Error-word bits of these calls (beside those of trellis.h). */
enum { TRELLIS_KV4_ERR_BAD = 4, TRELLIS_KV4_ERR_NO_PAGES = 8 };

/* A cache (passed by HOST pointer).  head_dim 128 or 256; page_size 16, 32, 64, 128 or 256;
 * 1 <= n_kv_heads <= 1024; pool 256-byte aligned. */
typedef struct {
  void *pool;
  int32_t n_layers;
  int32_t n_pages;
  int32_t page_size;
  int32_t n_kv_heads;
  int32_t head_dim;
} trellis_kv4_cache;

/* The sequences of a call (passed by HOST pointer): sequence b is slot slots[b] (slots NULL:
 * slot b) and has the rows cu[b] .. cu[b+1]-1 of the call's packed arrays, its LAST
 * n_b = cu[b+1] - cu[b] tokens: row cu[b] + i is the token at position lens[slot] - n_b + i.
 * lens already counts the call's new tokens (trellis_kv4_reserve adds them). */
typedef struct {
  const int32_t *table; /* [n_slots][max_pages] */
  const int32_t *lens;  /* [n_slots] */
  const int32_t *slots; /* [n_seq] or NULL */
  const int32_t *cu;    /* [n_seq + 1], cu[0] = 0, ascending, cu[n_seq] = rows */
  int32_t n_slots;
  int32_t max_pages;
  int32_t n_seq;
  int32_t rows;
} trellis_kv4_batch;

/* Bytes of one page of one layer (0 for sizes the format does not have). */
size_t trellis_kv4_page_bytes(int page_size, int n_kv_heads, int head_dim);

/* Workspace bytes: of append, read and free (any sizes) ... */
size_t trellis_kv4_workspace_bytes(void);
/* ... of attn with n_q_heads query heads (0 for invalid arguments) ... */
size_t trellis_kv4_attn_workspace_bytes(const trellis_kv4_cache *c, const trellis_kv4_batch *b, int n_q_heads);
/* ... of reserve, fork and compact over n slots (0 for invalid arguments). */
size_t trellis_kv4_pages_workspace_bytes(const trellis_kv4_cache *c, int n);

/* Quantise the batch's rows of new keys and values into one layer.
 * k, v: [rows][n_kv_heads][head_dim] of `dtype`, each head's vector contiguous, rows and heads
 * at the given strides (elements, multiples of 8; slices of a fused projection's output need no
 * copy), 16-byte aligned.  Pages that several slots hold must not be written (fork gives a
 * child its own last page).  One launch. */
int trellis_kv4_append(const trellis_kv4_cache *c, int layer, const trellis_kv4_batch *b, int dtype, const void *k,
                       int64_t k_row, int64_t k_head, const void *v, int64_t v_row, int64_t v_head, void *ws,
                       size_t ws_bytes, void *stream);

/* The keys and values that the cache holds for the batch's rows, rotated back:
 * k, v: out [rows][n_kv_heads][head_dim] of `dtype`, dense, 16-byte aligned.  One launch. */
int trellis_kv4_read(const trellis_kv4_cache *c, int layer, const trellis_kv4_batch *b, int dtype, void *k, void *v,
                     void *ws, size_t ws_bytes, void *stream);

/* Attention of the batch's rows over their sequences, causal:
 *   p = lens - n_b + i;  key j is visible iff j < lens, j <= p and
 *       (window == 0 or j > p - window or j < sinks)
 *   y = sum_j softmax_j(scale * q . k_j) v_j over the visible keys; no visible key: y = 0.
 * q  : [rows][n_q_heads][head_dim] of `dtype`, strides as for append; query head h reads key/
 *      value head h / (n_q_heads / n_kv_heads); n_q_heads is a multiple of n_kv_heads, at most
 *      64 times it.
 * y  : out [rows][n_q_heads][head_dim] of `dtype`, dense, 16-byte aligned; must not overlap q.
 * lse: NULL, or f32 out [rows][n_q_heads]: the natural logarithm of the softmax's denominator
 *      (-inf where no key is visible), by which results over parts of a context are joined.
 * A key whose weight is zero in fp32 adds nothing, whatever its value holds.  A weight times its value's
 * scale is held within 2^-11 of itself, but in steps of up to 2^-24 of the largest value scale that some
 * row of the call sees among its 128 tokens.
 * window >= 0 (0: none), sinks >= 0, scale finite.
 * max_rows: the caller's bound on n_b, 0 if unknown; it chooses kernels, results are right for
 *      any value.  One launch, two where some sequences may have few and others many rows. */
int trellis_kv4_attn(const trellis_kv4_cache *c, int layer, const trellis_kv4_batch *b, int dtype, const void *q,
                     int64_t q_row, int64_t q_head, int n_q_heads, float scale, int window, int sinks, int max_rows,
                     void *y, float *lse, void *ws, size_t ws_bytes, void *stream);

/* Make room: lens[slots[i]] += add[i] (>= 0) with the pages that takes, for i in [0, n);
 * slots distinct, or NULL (slot i).  Pages are taken lowest number first, in the order of i.
 * table int32 [n_slots][max_pages], lens int32 [n_slots], ref int32 [n_pages].  One launch. */
int trellis_kv4_reserve(const trellis_kv4_cache *c, int32_t *table, int32_t *lens, int n_slots, int max_pages,
                        int32_t *ref, const int32_t *slots, const int32_t *add, int n, void *ws, size_t ws_bytes,
                        void *stream);

/* Slot dst[i] becomes a copy of slot src[i], for i in [0, n): full pages are shared (ref + 1),
 * a last, partly filled page is copied into a page of its own (every layer's).  What dst held
 * is released.  dst distinct, none of them a src.  Two launches. */
int trellis_kv4_fork(const trellis_kv4_cache *c, int32_t *table, int32_t *lens, int n_slots, int max_pages,
                     int32_t *ref, const int32_t *src, const int32_t *dst, int n, void *ws, size_t ws_bytes,
                     void *stream);

/* Slot dst[i] becomes the tokens keep[keep_cu[i] .. keep_cu[i+1]-1] (positions in slot src[i],
 * in any order) packed into new pages of its own, every layer's.  What dst held is released.
 * dst distinct; dst[i] may be src[i] (in place), not another src.  n_keep = keep_cu[n], at most
 * 2^27.
 * Three launches. */
int trellis_kv4_compact(const trellis_kv4_cache *c, int32_t *table, int32_t *lens, int n_slots, int max_pages,
                        int32_t *ref, const int32_t *src, const int32_t *dst, int n, const int32_t *keep,
                        const int32_t *keep_cu, int n_keep, void *ws, size_t ws_bytes, void *stream);

/* Release slots[0 .. n): their pages' counts drop by one, their lengths become 0 (their table
 * rows are left).  A slot named twice is released once.  One launch (the list is checked before
 * anything is released). */
int trellis_kv4_free(const trellis_kv4_cache *c, const int32_t *table, int32_t *lens, int n_slots, int max_pages,
                     int32_t *ref, const int32_t *slots, int n, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TRELLIS_KV4_H_ */
