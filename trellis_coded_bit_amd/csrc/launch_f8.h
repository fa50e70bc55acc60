// Internal launchers behind include/trellis_f8.h and include/trellis_route.h.  Arguments are
// validated by api_f8.cpp.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/trellis_f8.h"
#include "../../include/trellis_route.h"

namespace trellis {

constexpr int kF8Block = 128;       // channels that share a scale
constexpr int kF8MaxNorm = 32768;   // channels of a norm's row, at most

// Rows quantised per block: q and scale, or y in 16 bits, or both.
struct F8RowsOut {
  uint8_t *q;
  float *scale;
  uint16_t *y;
};

struct F8Norm {
  int bf16;
  const uint16_t *x;
  int64_t x_row;
  const uint16_t *residual, *gamma;
  int rows, n;
  float eps;
  uint16_t *h;
  F8RowsOut out;
};
hipError_t launch_f8_norm(const F8Norm &a, hipStream_t stream);

struct F8Act {
  int bf16;
  const uint16_t *x;
  int64_t x_row;
  int rows, n;
  F8RowsOut out;
};
hipError_t launch_f8_silu_mul(const F8Act &a, hipStream_t stream);

// A product: one matrix (offsets NULL: all rows) or one per expert.
struct F8Gemm {
  trellis_f8_linear L;
  const uint8_t *q;
  const float *s;
  int64_t q_row, s_row;
  int n_q, rows;
  const int32_t *offsets, *order;
  int per;
  int bf16;
  uint16_t *y;
  int64_t y_row;
};
size_t f8_gemm_workspace_bytes(const trellis_f8_linear &L, int rows, bool grouped);
hipError_t launch_f8_gemm(const F8Gemm &a, void *ws, hipStream_t stream);

constexpr int kMoeExperts = 2048;  // of a sort, at most
size_t moe_sort_workspace_bytes(int tokens, int top, int n_experts);
hipError_t launch_moe_sort(const int32_t *ids, int tokens, int top, int n_experts, int32_t *offsets, int32_t *order,
                           int32_t *inverse, void *ws, hipStream_t stream);
hipError_t launch_moe_gather(const void *x, int64_t x_row_bytes, int tokens, int64_t row_bytes, const int32_t *order,
                             int rows, int per, void *out, uint32_t *errword, hipStream_t stream);

struct MoeCombine {
  int bf16;
  const uint16_t *y;      // combine: rows in; gradient: rows of the forward pass, or NULL
  const uint16_t *d_out;  // gradient
  int rows, n;
  const int32_t *inverse;
  const float *weights;
  int tokens, top;
  const uint16_t *add;  // combine
  uint16_t *out;        // combine: tokens; gradient: d_y
  float *d_weights;     // gradient
};
hipError_t launch_moe_combine(const MoeCombine &a, uint32_t *errword, hipStream_t stream);
hipError_t launch_moe_combine_grad(const MoeCombine &a, uint32_t *errword, hipStream_t stream);

}  // namespace trellis
