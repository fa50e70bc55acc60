// Products of block-scaled E4M3 rows with block-scaled E4M3 matrices, one or one per expert
// (include/trellis_f8.h).
//
// y[m][o] = sum over blocks b of 128 inputs of s[m][b] sw[o / 128][b] (q[m] . w[o] over the block):
// one v_mfma_f32_16x16x128_f8f6f4 forms a 16 x 16 tile of a block's products from zero, and a
// vector fma adds it times its scales.  Matrix rows are the tile's rows and tokens its columns, so
// a lane's four sums belong to one token and take one factor.
#include "f8_device.h"

namespace trellis {

namespace {

typedef int intx8 __attribute__((ext_vector_type(8)));

struct GemmArgs {
  F8Gemm g;
  uint32_t *errword;
  int kb;         // blocks of 128 inputs
  int col_tiles;  // tiles over out_features
  int row_tiles;  // tiles over rows, at most
};

// Which rows a tile of BM rows has: of expert e, rows [row, end).  e < 0: none.
struct RowTile {
  int e, row, end;
};

// Tile `at` of the list: every expert's rows in tiles of BM, expert after expert.  Called by whole
// waves; each lane looks at every 64th expert.  The list ends at the first pair of offsets that is
// out of order or out of range.
template <int BM>
__device__ __forceinline__ RowTile find_tile(const GemmArgs &p, int at, bool report) {
  if (!p.g.offsets) return {0, at * BM, p.g.rows};
  const int lane = threadIdx.x & 63, E = p.g.L.n_experts;
  if (ldg(p.g.offsets) != 0) {
    if (report && lane == 0) f8_error(p.errword);
    return {-1, 0, 0};
  }
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int a = 0, b = 0;
    if (e < E) {
      a = ldg(p.g.offsets + e);
      b = ldg(p.g.offsets + e + 1);
    }
    const uint64_t bad = __ballot(a < 0 || b < a || b > p.g.rows);
    const int good = bad ? __builtin_ctzll(bad) : 64;
    const int tiles = lane < good ? (b - a + BM - 1) / BM : 0;
    int s = tiles;
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(s, d, 64);
      if (lane >= d) s += o;
    }
    const uint64_t has = __ballot(at < s);
    if (has) {
      const int l = __builtin_ctzll(has);
      const int before = __shfl(s - tiles, l, 64);
      return {e0 + l, __shfl(a, l, 64) + (at - before) * BM, __shfl(b, l, 64)};
    }
    if (bad) {
      if (report && lane == 0) f8_error(p.errword);
      return {-1, 0, 0};
    }
    at -= __shfl(s, 63, 64);
  }
  return {-1, 0, 0};
}

// The row of q that a row reads, or -1.
__device__ __forceinline__ int source_row(const GemmArgs &p, int row) {
  if (!p.g.order) return row;
  const int entry = ldg(p.g.order + row);
  const int src = entry / p.g.per;
  if (entry < 0 || src >= p.g.n_q) {
    f8_error(p.errword);
    return -1;
  }
  return src;
}

template <bool BF>
__global__ __launch_bounds__(64) void simple_kernel(GemmArgs p) {
  const trellis_f8_linear &L = p.g.L;
  const int lane = threadIdx.x, i = lane & 15, g = lane >> 4;
  const int rt = blockIdx.x / p.col_tiles, ct = blockIdx.x - rt * p.col_tiles;
  const RowTile t = find_tile<16>(p, rt, rt == p.row_tiles - 1 && ct == 0);
  if (t.e < 0) return;
  const int K = L.in_features, N = L.out_features;
  const int row = t.row + i, o = ct * 16 + i;
  const bool live = row < t.end;
  const int src = live ? source_row(p, row) : -1;
  const uint8_t *x = p.g.q + (int64_t)max(src, 0) * p.g.q_row;
  const float *sx = p.g.s + (int64_t)max(src, 0) * p.g.s_row;
  const uint8_t *w = L.w + ((int64_t)t.e * N + min(o, N - 1)) * K;
  const float *sw = L.scale + ((int64_t)t.e * ((N + 127) / 128) + ct * 16 / 128) * p.kb;
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int b = 0; b < p.kb; ++b) {
    intx8 a8, b8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = b * 128 + h * 64 + 16 * g;
      u32x4 wv = ldg(reinterpret_cast<const u32x4 *>(w + min(k, K - 16)));
      u32x4 xv = ldg(reinterpret_cast<const u32x4 *>(x + min(k, K - 16)));
      if (k >= K) wv = xv = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a8[4 * h + j] = (int)wv[j];
        b8[4 * h + j] = (int)xv[j];
      }
    }
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    const floatx4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, zero, 0, 0, 0, 0, 0, 0);
    const float f = ldg(sx + b) * ldg(sw + b);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = fmaf(d[j], f, acc[j]);
  }
  if (!live) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = ct * 16 + 4 * g + j;
    if (c < N) stg(p.g.y + (int64_t)row * p.g.y_row + c, f8_narrow<BF>(src < 0 ? 0.f : acc[j]));
  }
}

}  // namespace

size_t f8_gemm_workspace_bytes(const trellis_f8_linear &L, int rows, bool grouped) { return kWsReserved; }

hipError_t launch_f8_gemm(const F8Gemm &a, void *ws, hipStream_t stream) {
  GemmArgs p{};
  p.g = a;
  p.errword = static_cast<uint32_t *>(ws);
  p.kb = (a.L.in_features + 127) / 128;
  p.col_tiles = (a.L.out_features + 15) / 16;
  p.row_tiles = a.offsets ? a.rows / 16 + min(a.rows, a.L.n_experts) : (a.rows + 15) / 16;
  const long long grid = (long long)p.row_tiles * p.col_tiles;
  if (a.bf16) simple_kernel<true><<<(unsigned)grid, 64, 0, stream>>>(p);
  else simple_kernel<false><<<(unsigned)grid, 64, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace trellis
