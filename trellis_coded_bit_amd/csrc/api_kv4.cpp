// C ABI of the 4-bit key/value cache: argument validation and dispatch.  The contract is in
// include/trellis_kv4.h.
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "../../include/trellis_kv4.h"
#include "abi.h"
#include "launch.h"
#include "launch_kv4.h"

using trellis::abi_clear;
using trellis::abi_fail;
using trellis::abi_hip_status;
using trellis::WorkspaceTurn;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

bool page_size_ok(int t) { return t == 16 || t == 32 || t == 64 || t == 128 || t == 256; }

int check_cache(const trellis_kv4_cache *c) {
  if (!c) return abi_fail(TRELLIS_EINVAL, "cache descriptor is NULL");
  if (trellis_kv4_page_bytes(c->page_size, c->n_kv_heads, c->head_dim) == 0)
    return abi_fail(TRELLIS_EINVAL,
                    "page_size=%d n_kv_heads=%d head_dim=%d: pages of 16, 32, 64, 128 or 256 tokens, 1..1024 heads of "
                    "128 or 256 expected",
                    c->page_size, c->n_kv_heads, c->head_dim);
  if (c->n_layers < 1 || c->n_pages < 1 || c->n_layers > 65535 || c->n_pages > (1 << 28))
    return abi_fail(TRELLIS_EINVAL, "n_layers=%d (1..65535), n_pages=%d (1..2^28)", c->n_layers, c->n_pages);
  if (!c->pool) return abi_fail(TRELLIS_EINVAL, "pool is NULL");
  if (!aligned(c->pool, 256)) return abi_fail(TRELLIS_EALIGN, "pool must be 256-byte aligned");
  return TRELLIS_OK;
}

int check_sizes(int n_slots, int max_pages, const trellis_kv4_cache *c) {
  if (n_slots < 1 || max_pages < 1) return abi_fail(TRELLIS_EINVAL, "n_slots=%d max_pages=%d must be positive", n_slots, max_pages);
  if ((long long)max_pages * c->page_size > (1LL << 29))
    return abi_fail(TRELLIS_EINVAL, "max_pages=%d pages of %d tokens exceed 2^29 tokens", max_pages, c->page_size);
  return TRELLIS_OK;
}

int check_batch(const trellis_kv4_cache *c, int layer, const trellis_kv4_batch *b, int dtype) {
  int st = check_cache(c);
  if (st) return st;
  if (!b) return abi_fail(TRELLIS_EINVAL, "batch descriptor is NULL");
  if (layer < 0 || layer >= c->n_layers) return abi_fail(TRELLIS_EINVAL, "layer=%d not in 0..%d", layer, c->n_layers - 1);
  if (dtype != TRELLIS_KV4_F16 && dtype != TRELLIS_KV4_BF16) return abi_fail(TRELLIS_EINVAL, "dtype=%d: 0 (fp16) or 1 (bf16) expected", dtype);
  if ((st = check_sizes(b->n_slots, b->max_pages, c))) return st;
  if (b->n_seq < 0 || b->rows < 0) return abi_fail(TRELLIS_EINVAL, "n_seq=%d rows=%d must not be negative", b->n_seq, b->rows);
  if (b->n_seq > (1 << 20) || b->rows > (1 << 26))
    return abi_fail(TRELLIS_EINVAL, "n_seq=%d (at most 2^20) or rows=%d (at most 2^26) too large", b->n_seq, b->rows);
  if (b->rows > 0 && b->n_seq == 0) return abi_fail(TRELLIS_EINVAL, "rows=%d without a sequence", b->rows);
  if (b->rows == 0) return TRELLIS_OK;
  if (!b->table || !b->lens || !b->cu) return abi_fail(TRELLIS_EINVAL, "table, lens or cu is NULL");
  if (!aligned(b->table, 4) || !aligned(b->lens, 4) || !aligned(b->cu, 4) || !aligned(b->slots, 4))
    return abi_fail(TRELLIS_EALIGN, "table, lens, cu and slots must be 4-byte aligned");
  return TRELLIS_OK;
}

int check_rows(const char *name, const void *p, int64_t row, int64_t head) {
  if (!p) return abi_fail(TRELLIS_EINVAL, "%s is NULL", name);
  if (!aligned(p, 16)) return abi_fail(TRELLIS_EALIGN, "%s must be 16-byte aligned", name);
  if (row < 0 || head < 0) return abi_fail(TRELLIS_EINVAL, "%s: negative strides (%lld, %lld)", name, (long long)row, (long long)head);
  if (row % 8 || head % 8) return abi_fail(TRELLIS_EALIGN, "%s: strides (%lld, %lld) must be multiples of 8 elements", name, (long long)row, (long long)head);
  return TRELLIS_OK;
}

int check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need || !aligned(ws, 256))
    return abi_fail(TRELLIS_EWORKSPACE, "workspace needs %zu bytes, 256-byte aligned (got %zu)", need, ws_bytes);
  return TRELLIS_OK;
}

int check_pages(const trellis_kv4_cache *c, const int32_t *table, const int32_t *lens, int n_slots, int max_pages,
                const int32_t *ref, int n) {
  int st = check_cache(c);
  if (st) return st;
  if ((st = check_sizes(n_slots, max_pages, c))) return st;
  // the plan keeps one bit per slot in shared memory
  if (n_slots > (1 << 18)) return abi_fail(TRELLIS_EINVAL, "n_slots=%d exceeds 2^18", n_slots);
  if (n < 0 || n > n_slots) return abi_fail(TRELLIS_EINVAL, "n=%d not in 0..n_slots=%d", n, n_slots);
  if (!table || !lens || !ref) return abi_fail(TRELLIS_EINVAL, "table, lens or ref is NULL");
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(ref, 4))
    return abi_fail(TRELLIS_EALIGN, "table, lens and ref must be 4-byte aligned");
  return TRELLIS_OK;
}

int check_list(const char *name, const int32_t *p) {
  if (!p) return abi_fail(TRELLIS_EINVAL, "%s is NULL", name);
  if (!aligned(p, 4)) return abi_fail(TRELLIS_EALIGN, "%s must be 4-byte aligned", name);
  return TRELLIS_OK;
}

trellis::Kv4Pages pages_of(const trellis_kv4_cache *c, int32_t *table, int32_t *lens, int n_slots, int max_pages,
                           int32_t *ref, int n) {
  trellis::Kv4Pages p{};
  p.c = *c;
  p.table = table;
  p.lens = lens;
  p.ref = ref;
  p.n_slots = n_slots;
  p.max_pages = max_pages;
  p.n = n;
  return p;
}

}  // namespace

extern "C" {

size_t trellis_kv4_page_bytes(int page_size, int n_kv_heads, int head_dim) {
  if (!page_size_ok(page_size) || n_kv_heads < 1 || n_kv_heads > 1024 || (head_dim != 128 && head_dim != 256)) return 0;
  return (size_t)132 * (head_dim / 128) * page_size * n_kv_heads;
}

size_t trellis_kv4_workspace_bytes(void) { return trellis::kWsReserved; }

size_t trellis_kv4_attn_workspace_bytes(const trellis_kv4_cache *c, const trellis_kv4_batch *b, int n_q_heads) {
  abi_clear();
  if (check_batch(c, 0, b, 0)) return 0;
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads || n_q_heads / c->n_kv_heads > 64) {
    abi_fail(TRELLIS_EINVAL, "n_q_heads=%d must be 1..64 times n_kv_heads=%d", n_q_heads, c->n_kv_heads);
    return 0;
  }
  return trellis::kv4_attn_workspace_bytes(*c, *b, n_q_heads);
}

size_t trellis_kv4_pages_workspace_bytes(const trellis_kv4_cache *c, int n) {
  abi_clear();
  if (!c || c->n_pages < 1 || n < 0) return 0;
  return trellis::kv4_pages_workspace_bytes(c->n_pages, n);
}

int trellis_kv4_append(const trellis_kv4_cache *c, int layer, const trellis_kv4_batch *b, int dtype, const void *k,
                       int64_t k_row, int64_t k_head, const void *v, int64_t v_row, int64_t v_head, void *ws,
                       size_t ws_bytes, void *stream) {
  abi_clear();
  int st = check_batch(c, layer, b, dtype);
  if (st) return st;
  if (b->rows == 0) return TRELLIS_OK;
  if ((st = check_rows("k", k, k_row, k_head)) || (st = check_rows("v", v, v_row, v_head))) return st;
  if ((st = check_ws(ws, ws_bytes, trellis::kWsReserved))) return st;
  return abi_hip_status(trellis::launch_kv4_append(*c, layer, *b, dtype, {k, k_row, k_head}, {v, v_row, v_head},
                                                   static_cast<uint32_t *>(ws), as_stream(stream)),
                        "trellis_kv4_append launch");
}

int trellis_kv4_read(const trellis_kv4_cache *c, int layer, const trellis_kv4_batch *b, int dtype, void *k, void *v,
                     void *ws, size_t ws_bytes, void *stream) {
  abi_clear();
  int st = check_batch(c, layer, b, dtype);
  if (st) return st;
  if (b->rows == 0) return TRELLIS_OK;
  if ((st = check_rows("k", k, 0, 0)) || (st = check_rows("v", v, 0, 0))) return st;
  if ((st = check_ws(ws, ws_bytes, trellis::kWsReserved))) return st;
  return abi_hip_status(trellis::launch_kv4_read(*c, layer, *b, dtype, k, v, static_cast<uint32_t *>(ws), as_stream(stream)),
                        "trellis_kv4_read launch");
}

int trellis_kv4_attn(const trellis_kv4_cache *c, int layer, const trellis_kv4_batch *b, int dtype, const void *q,
                     int64_t q_row, int64_t q_head, int n_q_heads, float scale, int window, int sinks, int max_rows,
                     void *y, float *lse, void *ws, size_t ws_bytes, void *stream) {
  abi_clear();
  int st = check_batch(c, layer, b, dtype);
  if (st) return st;
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads || n_q_heads / c->n_kv_heads > 64)
    return abi_fail(TRELLIS_EINVAL, "n_q_heads=%d must be 1..64 times n_kv_heads=%d", n_q_heads, c->n_kv_heads);
  if ((long long)b->rows * n_q_heads > (1LL << 30))
    return abi_fail(TRELLIS_EINVAL, "rows=%d times n_q_heads=%d exceed 2^30", b->rows, n_q_heads);
  if (window < 0 || sinks < 0 || max_rows < 0)
    return abi_fail(TRELLIS_EINVAL, "window=%d sinks=%d max_rows=%d must not be negative", window, sinks, max_rows);
  if (!std::isfinite(scale)) return abi_fail(TRELLIS_EINVAL, "scale must be finite");
  if (b->rows == 0) return TRELLIS_OK;
  if ((st = check_rows("q", q, q_row, q_head)) || (st = check_rows("y", y, 0, 0))) return st;
  if (!aligned(lse, 4)) return abi_fail(TRELLIS_EALIGN, "lse must be 4-byte aligned");
  // workgroups write rows of y while others still read rows of q
  const char *q0 = static_cast<const char *>(q), *y0 = static_cast<const char *>(y);
  const size_t q_bytes = 2 * ((size_t)(b->rows - 1) * q_row + (size_t)(n_q_heads - 1) * q_head + c->head_dim);
  const size_t y_bytes = (size_t)2 * b->rows * n_q_heads * c->head_dim;
  if (q0 < y0 + y_bytes && y0 < q0 + q_bytes) return abi_fail(TRELLIS_EINVAL, "y overlaps q");
  if ((st = check_ws(ws, ws_bytes, trellis::kv4_attn_workspace_bytes(*c, *b, n_q_heads)))) return st;
  trellis::Kv4Attn a{};
  a.c = *c;
  a.b = *b;
  a.layer = layer;
  a.dtype = dtype;
  a.n_q_heads = n_q_heads;
  a.window = window;
  a.sinks = sinks;
  a.max_rows = max_rows;
  a.q = {q, q_row, q_head};
  a.scale = scale;
  a.y = y;
  a.lse = lse;
  const WorkspaceTurn turn(ws);
  return abi_hip_status(trellis::launch_kv4_attn(a, ws, as_stream(stream)), "trellis_kv4_attn launch");
}

int trellis_kv4_reserve(const trellis_kv4_cache *c, int32_t *table, int32_t *lens, int n_slots, int max_pages,
                        int32_t *ref, const int32_t *slots, const int32_t *add, int n, void *ws, size_t ws_bytes,
                        void *stream) {
  abi_clear();
  int st = check_pages(c, table, lens, n_slots, max_pages, ref, n);
  if (st) return st;
  if (n == 0) return TRELLIS_OK;
  if ((st = check_list("add", add))) return st;
  if (!aligned(slots, 4)) return abi_fail(TRELLIS_EALIGN, "slots must be 4-byte aligned");
  if ((st = check_ws(ws, ws_bytes, trellis::kv4_pages_workspace_bytes(c->n_pages, n)))) return st;
  trellis::Kv4Pages p = pages_of(c, table, lens, n_slots, max_pages, ref, n);
  p.dst = slots;
  p.add = add;
  const WorkspaceTurn turn(ws);
  return abi_hip_status(trellis::launch_kv4_reserve(p, ws, as_stream(stream)), "trellis_kv4_reserve launch");
}

int trellis_kv4_fork(const trellis_kv4_cache *c, int32_t *table, int32_t *lens, int n_slots, int max_pages,
                     int32_t *ref, const int32_t *src, const int32_t *dst, int n, void *ws, size_t ws_bytes,
                     void *stream) {
  abi_clear();
  int st = check_pages(c, table, lens, n_slots, max_pages, ref, n);
  if (st) return st;
  if (n == 0) return TRELLIS_OK;
  if ((st = check_list("src", src)) || (st = check_list("dst", dst))) return st;
  if ((st = check_ws(ws, ws_bytes, trellis::kv4_pages_workspace_bytes(c->n_pages, n)))) return st;
  trellis::Kv4Pages p = pages_of(c, table, lens, n_slots, max_pages, ref, n);
  p.src = src;
  p.dst = dst;
  const WorkspaceTurn turn(ws);
  return abi_hip_status(trellis::launch_kv4_fork(p, ws, as_stream(stream)), "trellis_kv4_fork launch");
}

int trellis_kv4_compact(const trellis_kv4_cache *c, int32_t *table, int32_t *lens, int n_slots, int max_pages,
                        int32_t *ref, const int32_t *src, const int32_t *dst, int n, const int32_t *keep,
                        const int32_t *keep_cu, int n_keep, void *ws, size_t ws_bytes, void *stream) {
  abi_clear();
  int st = check_pages(c, table, lens, n_slots, max_pages, ref, n);
  if (st) return st;
  if (n_keep < 0 || n_keep > trellis::kKv4MaxKeep)
    return abi_fail(TRELLIS_EINVAL, "n_keep=%d not in 0..%d", n_keep, trellis::kKv4MaxKeep);
  if (n == 0) return TRELLIS_OK;
  if ((st = check_list("src", src)) || (st = check_list("dst", dst)) || (st = check_list("keep_cu", keep_cu))) return st;
  if (n_keep > 0 && (st = check_list("keep", keep))) return st;
  if ((st = check_ws(ws, ws_bytes, trellis::kv4_pages_workspace_bytes(c->n_pages, n)))) return st;
  trellis::Kv4Pages p = pages_of(c, table, lens, n_slots, max_pages, ref, n);
  p.src = src;
  p.dst = dst;
  p.keep = keep;
  p.keep_cu = keep_cu;
  p.n_keep = n_keep;
  const WorkspaceTurn turn(ws);
  return abi_hip_status(trellis::launch_kv4_compact(p, ws, as_stream(stream)), "trellis_kv4_compact launch");
}

int trellis_kv4_free(const trellis_kv4_cache *c, const int32_t *table, int32_t *lens, int n_slots, int max_pages,
                     int32_t *ref, const int32_t *slots, int n, void *ws, size_t ws_bytes, void *stream) {
  abi_clear();
  int st = check_pages(c, table, lens, n_slots, max_pages, ref, n);
  if (st) return st;
  if (n == 0) return TRELLIS_OK;
  if ((st = check_list("slots", slots))) return st;
  if ((st = check_ws(ws, ws_bytes, trellis::kWsReserved))) return st;
  trellis::Kv4Pages p = pages_of(c, const_cast<int32_t *>(table), lens, n_slots, max_pages, ref, n);
  p.dst = slots;
  return abi_hip_status(trellis::launch_kv4_free(p, static_cast<uint32_t *>(ws), as_stream(stream)),
                        "trellis_kv4_free launch");
}

}  // extern "C"
