// Internal launchers behind include/trellis_kv4.h.  Arguments are validated by api_kv4.cpp.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/trellis_kv4.h"

namespace trellis {

// Rows of strided vectors: element (row, head, d) at row * row_stride + head * head_stride + d.
struct Kv4Rows {
  const void *p;
  int64_t row_stride, head_stride;
};

hipError_t launch_kv4_append(const trellis_kv4_cache &c, int layer, const trellis_kv4_batch &b, int dtype,
                             const Kv4Rows &k, const Kv4Rows &v, uint32_t *errword, hipStream_t stream);
hipError_t launch_kv4_read(const trellis_kv4_cache &c, int layer, const trellis_kv4_batch &b, int dtype, void *k,
                           void *v, uint32_t *errword, hipStream_t stream);

struct Kv4Attn {
  trellis_kv4_cache c;
  trellis_kv4_batch b;
  int layer, dtype, n_q_heads, window, sinks, max_rows;
  Kv4Rows q;
  float scale;
  void *y;
  float *lse;
};
size_t kv4_attn_workspace_bytes(const trellis_kv4_cache &c, const trellis_kv4_batch &b, int n_q_heads);
hipError_t launch_kv4_attn(const Kv4Attn &a, void *ws, hipStream_t stream);

// The page operations' state and items.
struct Kv4Pages {
  trellis_kv4_cache c;
  int32_t *table, *lens, *ref;
  int n_slots, max_pages, n;
  const int32_t *src, *dst;       // fork, compact; reserve: dst = slots (or NULL)
  const int32_t *add;             // reserve
  const int32_t *keep, *keep_cu;  // compact
  int n_keep;
};
// Tokens that one compaction keeps, at most: 16 threads each, in a grid of less than 2^32.
constexpr int kKv4MaxKeep = 1 << 27;
size_t kv4_pages_workspace_bytes(int n_pages, int n);
hipError_t launch_kv4_reserve(const Kv4Pages &p, void *ws, hipStream_t stream);
hipError_t launch_kv4_fork(const Kv4Pages &p, void *ws, hipStream_t stream);
hipError_t launch_kv4_compact(const Kv4Pages &p, void *ws, hipStream_t stream);
hipError_t launch_kv4_free(const Kv4Pages &p, uint32_t *errword, hipStream_t stream);

}  // namespace trellis
