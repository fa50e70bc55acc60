// C ABI of the block-scaled FP8 operators and of the routed tokens: argument validation and
// dispatch.  The contracts are in include/trellis_f8.h and include/trellis_route.h.
#include <hip/hip_runtime_api.h>

#include <cfloat>
#include <cmath>
#include <initializer_list>

#include "../../include/trellis_f8.h"
#include "../../include/trellis_route.h"
#include "abi.h"
#include "launch.h"
#include "launch_f8.h"

using trellis::abi_clear;
using trellis::abi_fail;
using trellis::abi_hip_status;
using trellis::WorkspaceTurn;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

// Bytes that a call reads or writes.
struct Span {
  const char *name;
  const void *p;
  size_t bytes;
};
Span rows_span(const char *name, const void *p, int64_t rows, int64_t stride, int64_t row, size_t elem) {
  return {name, p, p && rows > 0 ? (size_t)((rows - 1) * stride + row) * elem : 0};
}
bool overlap(const Span &a, const Span &b) {
  if (!a.bytes || !b.bytes) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}
// No output may overlap another or an input.
int check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span *o = outs.begin(); o != outs.end(); ++o) {
    for (const Span *q = outs.begin(); q != o; ++q)
      if (overlap(*o, *q)) return abi_fail(TRELLIS_EINVAL, "%s overlaps %s", o->name, q->name);
    for (const Span &i : ins)
      if (overlap(*o, i)) return abi_fail(TRELLIS_EINVAL, "%s overlaps %s", o->name, i.name);
  }
  return TRELLIS_OK;
}

int check_dtype(int dtype) {
  if (dtype != TRELLIS_F8_F16 && dtype != TRELLIS_F8_BF16) return abi_fail(TRELLIS_EINVAL, "dtype=%d: 0 (fp16) or 1 (bf16) expected", dtype);
  return TRELLIS_OK;
}

int check_16(const char *name, const void *p) {
  if (!p) return abi_fail(TRELLIS_EINVAL, "%s is NULL", name);
  if (!aligned(p, 16)) return abi_fail(TRELLIS_EALIGN, "%s must be 16-byte aligned", name);
  return TRELLIS_OK;
}

int check_4(const char *name, const void *p) {
  if (!p) return abi_fail(TRELLIS_EINVAL, "%s is NULL", name);
  if (!aligned(p, 4)) return abi_fail(TRELLIS_EALIGN, "%s must be 4-byte aligned", name);
  return TRELLIS_OK;
}

int check_stride(const char *name, int64_t stride, int64_t least, int64_t unit, int64_t rows) {
  if (rows < 2) return TRELLIS_OK;  // (used for nothing)
  if (stride < least) return abi_fail(TRELLIS_EINVAL, "%s: row stride %lld below the row's %lld", name, (long long)stride, (long long)least);
  if (stride > (1LL << 40)) return abi_fail(TRELLIS_EINVAL, "%s: row stride %lld above 2^40", name, (long long)stride);
  if (stride % unit) return abi_fail(TRELLIS_EALIGN, "%s: row stride %lld must be a multiple of %lld", name, (long long)stride, (long long)unit);
  return TRELLIS_OK;
}

int check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need || !aligned(ws, 256))
    return abi_fail(TRELLIS_EWORKSPACE, "workspace needs %zu bytes, 256-byte aligned (got %zu)", need, ws_bytes);
  return TRELLIS_OK;
}

// The quantised rows' outputs.
int check_rows_out(const uint8_t *q, const float *scale, const void *y) {
  if (!q && !y) return abi_fail(TRELLIS_EINVAL, "q and y are both NULL");
  if ((q == nullptr) != (scale == nullptr)) return abi_fail(TRELLIS_EINVAL, "q and scale: both or neither");
  int st;
  if (q && ((st = check_16("q", q)) || (st = check_4("scale", scale)))) return st;
  return y ? check_16("y", y) : TRELLIS_OK;
}

int64_t blocks_of(int64_t n) { return (n + trellis::kF8Block - 1) / trellis::kF8Block; }

int check_linear(const trellis_f8_linear *L, bool one) {
  if (!L) return abi_fail(TRELLIS_EINVAL, "matrix descriptor is NULL");
  if (L->n_experts < 1 || L->n_experts > (1 << 16) || (one && L->n_experts != 1))
    return abi_fail(TRELLIS_EINVAL, "n_experts=%d: %s expected", L->n_experts, one ? "1" : "1..65536");
  if (L->in_features < 16 || L->in_features % 16 || L->in_features > (1 << 20) || L->out_features < 1 || L->out_features > (1 << 20))
    return abi_fail(TRELLIS_EINVAL, "in_features=%d (a multiple of 16, 16..2^20), out_features=%d (1..2^20)", L->in_features, L->out_features);
  return TRELLIS_OK;
}

int check_product(const trellis_f8_linear *L, bool one, int rows) {
  int st = check_linear(L, one);
  if (st) return st;
  if (rows < 0 || rows > (1 << 26)) return abi_fail(TRELLIS_EINVAL, "rows=%d not in 0..2^26", rows);
  // tiles of 16 x 16 at the least, in one grid
  if (((long long)rows / 16 + L->n_experts) * ((L->out_features + 15) / 16) >= (1LL << 31))
    return abi_fail(TRELLIS_EINVAL, "rows=%d times out_features=%d: more tiles than a launch holds", rows, L->out_features);
  return TRELLIS_OK;
}

int product(trellis::F8Gemm &a, int n_q, const char *what, void *ws, size_t ws_bytes, void *stream) {
  const int64_t k = a.L.in_features, n = a.L.out_features, kb = blocks_of(k), nb = blocks_of(n);
  int st;
  if ((st = check_16("w", a.L.w)) || (st = check_4("matrix scale", a.L.scale)) || (st = check_16("q", a.q)) || (st = check_4("s", a.s)))
    return st;
  if ((st = check_stride("q", a.q_row, k, 16, n_q)) || (st = check_stride("s", a.s_row, kb, 1, n_q))) return st;
  // the kernels count q's bytes from its start in 32 bits of 16
  if (n_q > 1 && a.q_row > (1LL << 36) / n_q)
    return abi_fail(TRELLIS_EINVAL, "q: %d rows at a stride of %lld bytes exceed 2^36", n_q, (long long)a.q_row);
  if (!a.y) return abi_fail(TRELLIS_EINVAL, "y is NULL");
  if (!aligned(a.y, 2)) return abi_fail(TRELLIS_EALIGN, "y must be 2-byte aligned");
  if ((st = check_stride("y", a.y_row, n, 1, a.rows))) return st;
  if (n_q < 2) a.q_row = a.s_row = 0;
  if (a.rows < 2) a.y_row = 0;
  if ((st = check_apart({rows_span("y", a.y, a.rows, a.y_row, n, 2)},
                        {rows_span("q", a.q, n_q, a.q_row, k, 1), rows_span("s", a.s, n_q, a.s_row, kb, 4),
                         {"w", a.L.w, (size_t)(a.L.n_experts * n * k)}, {"matrix scale", a.L.scale, (size_t)(a.L.n_experts * nb * kb * 4)},
                         {"offsets", a.offsets, a.offsets ? (size_t)4 * (a.L.n_experts + 1) : 0},
                         {"order", a.order, a.order ? (size_t)4 * a.rows : 0}})))
    return st;
  if ((st = check_ws(ws, ws_bytes, trellis::f8_gemm_workspace_bytes(a.L, a.rows, a.offsets != nullptr)))) return st;
  const WorkspaceTurn turn(ws);
  return abi_hip_status(trellis::launch_f8_gemm(a, ws, as_stream(stream)), what);
}

int check_route(int tokens, int top) {
  if (tokens < 0 || top < 1 || top > 1024 || (long long)tokens * top > (1 << 24))
    return abi_fail(TRELLIS_EINVAL, "tokens=%d top=%d: top in 1..1024 and at most 2^24 entries expected", tokens, top);
  return TRELLIS_OK;
}

int check_combine(int dtype, const void *y, int rows, int n, const int32_t *inverse, const float *weights, int tokens, int top) {
  int st = check_dtype(dtype);
  if (st || (st = check_route(tokens, top))) return st;
  if (rows < 0 || rows > (1 << 26)) return abi_fail(TRELLIS_EINVAL, "rows=%d not in 0..2^26", rows);
  if (n < 8 || n % 8 || n > (1 << 20)) return abi_fail(TRELLIS_EINVAL, "n=%d must be a multiple of 8 in 8..2^20", n);
  if (tokens == 0) return TRELLIS_OK;
  if (rows > 0 && (st = check_16("y", y))) return st;
  if ((st = check_4("inverse", inverse))) return st;
  if (!aligned(weights, 4)) return abi_fail(TRELLIS_EALIGN, "weights must be 4-byte aligned");
  return TRELLIS_OK;
}

}  // namespace

extern "C" {

int trellis_f8_norm(int dtype, const void *x, int64_t x_row, const void *residual, const void *gamma, int rows, int n,
                    float eps, void *h_out, uint8_t *q, float *scale, void *y, void *stream) {
  abi_clear();
  int st = check_dtype(dtype);
  if (st) return st;
  // (a workgroup of up to 1024 threads a row, below 2^32 threads in all)
  if (rows < 0 || rows >= (1 << 22)) return abi_fail(TRELLIS_EINVAL, "rows=%d not in 0..2^22-1", rows);
  if (n < 16 || n % 16 || n > trellis::kF8MaxNorm)
    return abi_fail(TRELLIS_EINVAL, "n=%d must be a multiple of 16 in 16..%d", n, trellis::kF8MaxNorm);
  if (!std::isfinite(eps) || eps < FLT_MIN) return abi_fail(TRELLIS_EINVAL, "eps=%g must be a normal positive number", (double)eps);
  if (rows == 0) return TRELLIS_OK;
  if ((st = check_16("x", x)) || (st = check_rows_out(q, scale, y))) return st;
  if ((st = check_stride("x", x_row, n, 8, rows))) return st;
  if (rows < 2) x_row = n;
  if ((residual && (st = check_16("residual", residual))) || (gamma && (st = check_16("gamma", gamma))) ||
      (h_out && (st = check_16("h_out", h_out))))
    return st;
  const Span sx = rows_span("x", x, rows, x_row, n, 2), sr = rows_span("residual", residual, rows, n, n, 2),
             sg = rows_span("gamma", gamma, 1, n, n, 2), sh = rows_span("h_out", h_out, rows, n, n, 2),
             sy = rows_span("y", y, rows, n, n, 2), sq = rows_span("q", q, rows, n, n, 1),
             ss = rows_span("scale", scale, rows, blocks_of(n), blocks_of(n), 4);
  if ((st = check_apart({sy, sq, ss}, {sx, sr, sg, sh})) || (st = check_apart({sh}, {sg}))) return st;
  if (h_out && ((!(h_out == x && x_row == n) && (st = check_apart({sh}, {sx}))) || (h_out != residual && (st = check_apart({sh}, {sr})))))
    return st;
  trellis::F8Norm a{};
  a.bf16 = dtype;
  a.x = static_cast<const uint16_t *>(x);
  a.x_row = x_row;
  a.residual = static_cast<const uint16_t *>(residual);
  a.gamma = static_cast<const uint16_t *>(gamma);
  a.rows = rows;
  a.n = n;
  a.eps = eps;
  a.h = static_cast<uint16_t *>(h_out);
  a.out = {q, scale, static_cast<uint16_t *>(y)};
  return abi_hip_status(trellis::launch_f8_norm(a, as_stream(stream)), "trellis_f8_norm launch");
}

int trellis_f8_silu_mul(int dtype, const void *x, int64_t x_row, int rows, int n, uint8_t *q, float *scale, void *y,
                        void *stream) {
  abi_clear();
  int st = check_dtype(dtype);
  if (st) return st;
  if (n < 16 || n % 16 || n > (1 << 20)) return abi_fail(TRELLIS_EINVAL, "n=%d must be a multiple of 16 in 16..2^20", n);
  if (rows < 0 || (int64_t)rows * blocks_of(n) > (1LL << 30))
    return abi_fail(TRELLIS_EINVAL, "rows=%d times n=%d not in 0..2^37", rows, n);
  if (rows == 0) return TRELLIS_OK;
  if ((st = check_16("x", x)) || (st = check_rows_out(q, scale, y))) return st;
  if ((st = check_stride("x", x_row, 2 * (int64_t)n, 8, rows))) return st;
  if (rows < 2) x_row = 2 * (int64_t)n;
  if ((st = check_apart({rows_span("y", y, rows, n, n, 2), rows_span("q", q, rows, n, n, 1),
                         rows_span("scale", scale, rows, blocks_of(n), blocks_of(n), 4)},
                        {rows_span("x", x, rows, x_row, 2 * (int64_t)n, 2)})))
    return st;
  trellis::F8Act a{dtype, static_cast<const uint16_t *>(x), x_row, rows, n, {q, scale, static_cast<uint16_t *>(y)}};
  return abi_hip_status(trellis::launch_f8_silu_mul(a, as_stream(stream)), "trellis_f8_silu_mul launch");
}

size_t trellis_f8_gemm_workspace_bytes(const trellis_f8_linear *L, int M) {
  abi_clear();
  return check_product(L, true, M) ? 0 : trellis::f8_gemm_workspace_bytes(*L, M, false);
}

size_t trellis_f8_moe_gemm_workspace_bytes(const trellis_f8_linear *L, int rows) {
  abi_clear();
  return check_product(L, false, rows) ? 0 : trellis::f8_gemm_workspace_bytes(*L, rows, true);
}

int trellis_f8_gemm(const trellis_f8_linear *L, const uint8_t *q, int64_t q_row, const float *s, int64_t s_row, int M,
                    int dtype, void *y, int64_t y_row, void *ws, size_t ws_bytes, void *stream) {
  abi_clear();
  int st = check_product(L, true, M);
  if (st || (st = check_dtype(dtype))) return st;
  if (M == 0) return TRELLIS_OK;
  trellis::F8Gemm a{*L, q, s, q_row, s_row, M, M, nullptr, nullptr, 1, dtype, static_cast<uint16_t *>(y), y_row};
  return product(a, M, "trellis_f8_gemm launch", ws, ws_bytes, stream);
}

int trellis_f8_moe_gemm(const trellis_f8_linear *L, const uint8_t *q, int64_t q_row, const float *s, int64_t s_row,
                        int n_q, const int32_t *offsets, const int32_t *order, int per, int rows, int dtype, void *y,
                        int64_t y_row, void *ws, size_t ws_bytes, void *stream) {
  abi_clear();
  int st = check_product(L, false, rows);
  if (st || (st = check_dtype(dtype))) return st;
  if (per < 1) return abi_fail(TRELLIS_EINVAL, "per=%d must be positive", per);
  if (n_q < 0 || n_q > (1 << 26) || (!order && n_q < rows)) return abi_fail(TRELLIS_EINVAL, "n_q=%d rows of q for rows=%d", n_q, rows);
  if (rows == 0) return TRELLIS_OK;
  if (n_q == 0) return abi_fail(TRELLIS_EINVAL, "n_q=0 rows of q for rows=%d", rows);
  if ((st = check_4("offsets", offsets))) return st;
  if (!aligned(order, 4)) return abi_fail(TRELLIS_EALIGN, "order must be 4-byte aligned");
  trellis::F8Gemm a{*L, q, s, q_row, s_row, n_q, rows, offsets, order, per, dtype, static_cast<uint16_t *>(y), y_row};
  return product(a, n_q, "trellis_f8_moe_gemm launch", ws, ws_bytes, stream);
}

size_t trellis_moe_sort_workspace_bytes(int tokens, int top, int n_experts) {
  abi_clear();
  if (check_route(tokens, top) || n_experts < 1 || n_experts > trellis::kMoeExperts) return 0;
  return trellis::moe_sort_workspace_bytes(tokens, top, n_experts);
}

size_t trellis_moe_rows_workspace_bytes(void) { return trellis::kWsReserved; }

int trellis_moe_sort(const int32_t *ids, int tokens, int top, int n_experts, int32_t *offsets, int32_t *order,
                     int32_t *inverse, void *ws, size_t ws_bytes, void *stream) {
  abi_clear();
  int st = check_route(tokens, top);
  if (st) return st;
  if (n_experts < 1 || n_experts > trellis::kMoeExperts)
    return abi_fail(TRELLIS_EINVAL, "n_experts=%d not in 1..%d", n_experts, trellis::kMoeExperts);
  if ((st = check_4("offsets", offsets))) return st;
  if (tokens > 0 && ((st = check_4("ids", ids)) || (st = check_4("order", order)) || (st = check_4("inverse", inverse)))) return st;
  const size_t entries = (size_t)4 * tokens * top;
  if ((st = check_apart({{"offsets", offsets, (size_t)4 * (n_experts + 1)}, {"order", order, entries}, {"inverse", inverse, entries}},
                        {{"ids", ids, entries}})))
    return st;
  if ((st = check_ws(ws, ws_bytes, trellis::moe_sort_workspace_bytes(tokens, top, n_experts)))) return st;
  const WorkspaceTurn turn(ws);
  return abi_hip_status(trellis::launch_moe_sort(ids, tokens, top, n_experts, offsets, order, inverse, ws, as_stream(stream)),
                        "trellis_moe_sort launch");
}

int trellis_moe_gather(const void *x, int64_t x_row_bytes, int tokens, int64_t row_bytes, const int32_t *order, int rows,
                       int per, void *out, void *ws, size_t ws_bytes, void *stream) {
  abi_clear();
  if (tokens < 0 || tokens > (1 << 26) || rows < 0 || rows > (1 << 26) || per < 1)
    return abi_fail(TRELLIS_EINVAL, "tokens=%d rows=%d (0..2^26), per=%d (positive)", tokens, rows, per);
  if (row_bytes < 4 || row_bytes % 4 || row_bytes > (1LL << 24))
    return abi_fail(TRELLIS_EINVAL, "row_bytes=%lld must be a multiple of 4 in 4..2^24", (long long)row_bytes);
  if (rows == 0) return TRELLIS_OK;
  int st;
  if ((tokens > 0 && (st = check_4("x", x))) || (st = check_4("order", order)) || (st = check_4("out", out))) return st;
  if ((st = check_stride("x", x_row_bytes, row_bytes, 4, tokens))) return st;
  if (tokens < 2) x_row_bytes = row_bytes;
  if ((st = check_apart({rows_span("out", out, rows, row_bytes, row_bytes, 1)},
                        {rows_span("x", x, tokens, x_row_bytes, row_bytes, 1), {"order", order, (size_t)4 * rows}})))
    return st;
  if ((st = check_ws(ws, ws_bytes, trellis::kWsReserved))) return st;
  return abi_hip_status(trellis::launch_moe_gather(x, x_row_bytes, tokens, row_bytes, order, rows, per, out,
                                                   static_cast<uint32_t *>(ws), as_stream(stream)),
                        "trellis_moe_gather launch");
}

int trellis_moe_combine(int dtype, const void *y, int rows, int n, const int32_t *inverse, const float *weights,
                        int tokens, int top, const void *add, void *out, void *ws, size_t ws_bytes, void *stream) {
  abi_clear();
  int st = check_combine(dtype, y, rows, n, inverse, weights, tokens, top);
  if (st) return st;
  if (tokens == 0) return TRELLIS_OK;
  if ((add && (st = check_16("add", add))) || (st = check_16("out", out))) return st;
  const size_t entries = (size_t)4 * tokens * top;
  const Span so = rows_span("out", out, tokens, n, n, 2), sa = rows_span("add", add, tokens, n, n, 2);
  if ((st = check_apart({so}, {rows_span("y", y, rows, n, n, 2), {"inverse", inverse, entries}, {"weights", weights, weights ? entries : 0}})) ||
      (add != out && (st = check_apart({so}, {sa}))))
    return st;
  if ((st = check_ws(ws, ws_bytes, trellis::kWsReserved))) return st;
  trellis::MoeCombine a{};
  a.bf16 = dtype;
  a.y = static_cast<const uint16_t *>(y);
  a.rows = rows;
  a.n = n;
  a.inverse = inverse;
  a.weights = weights;
  a.tokens = tokens;
  a.top = top;
  a.add = static_cast<const uint16_t *>(add);
  a.out = static_cast<uint16_t *>(out);
  return abi_hip_status(trellis::launch_moe_combine(a, static_cast<uint32_t *>(ws), as_stream(stream)), "trellis_moe_combine launch");
}

int trellis_moe_combine_grad(int dtype, const void *d_out, const void *y, int rows, int n, const int32_t *inverse,
                             const float *weights, int tokens, int top, void *d_y, float *d_weights, void *ws,
                             size_t ws_bytes, void *stream) {
  abi_clear();
  int st = check_combine(dtype, d_weights ? y : d_y, rows, n, inverse, weights, tokens, top);
  if (st) return st;
  if (tokens == 0) return TRELLIS_OK;
  if ((st = check_16("d_out", d_out)) || (rows > 0 && (st = check_16("d_y", d_y)))) return st;
  if (!aligned(d_weights, 4)) return abi_fail(TRELLIS_EALIGN, "d_weights must be 4-byte aligned");
  const size_t entries = (size_t)4 * tokens * top;
  const Span sy = rows_span("y", d_weights ? y : nullptr, rows, n, n, 2), sd = rows_span("d_y", d_y, rows, n, n, 2),
             sw = {"d_weights", d_weights, d_weights ? entries : 0};
  const Span so = rows_span("d_out", d_out, tokens, n, n, 2), si = {"inverse", inverse, entries}, sf = {"weights", weights, weights ? entries : 0};
  if ((st = check_apart({sd, sw}, {so, si, sf})) || (st = check_apart({sw}, {sy})) || (d_y != y && (st = check_apart({sd}, {sy})))) return st;
  if ((st = check_ws(ws, ws_bytes, trellis::kWsReserved))) return st;
  trellis::MoeCombine a{};
  a.bf16 = dtype;
  a.y = static_cast<const uint16_t *>(y);
  a.d_out = static_cast<const uint16_t *>(d_out);
  a.rows = rows;
  a.n = n;
  a.inverse = inverse;
  a.weights = weights;
  a.tokens = tokens;
  a.top = top;
  a.out = static_cast<uint16_t *>(d_y);
  a.d_weights = d_weights;
  return abi_hip_status(trellis::launch_moe_combine_grad(a, static_cast<uint32_t *>(ws), as_stream(stream)),
                        "trellis_moe_combine_grad launch");
}

}  // extern "C"
