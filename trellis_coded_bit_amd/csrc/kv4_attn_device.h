// What the attention kernels over the 4-bit cache share (their mathematics: kv4_attn.hip).
#pragma once
#include "kv4_device.h"

namespace trellis {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef short v2s __attribute__((ext_vector_type(2)));

constexpr int kTile = 128;  // keys of a tile: the depth of one matrix instruction
constexpr int kCols = 16;   // (row, head) pairs of a tile: its width
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();

struct AttnArgs {
  Kv4Attn a;
  uint32_t *errword;
  uint32_t *counters;  // one per workgroup, zero between calls
  int few;             // sequences of at most so many columns are the narrow kernel's, others the wide one's
  int tends;           // this launch checks the sequences and clears the rows that none has
  int splits;          // wide: workgroups that share a segment
  float *parts;        // [workgroups][2][C][D + 8]: unnormalised sums, then maximum, sum of weights
  int group;           // query heads per key/value head
  uint32_t per_group;  // 65536 / group + 1: x * per_group >> 16 is x / group up to x = 255
  int page_shift;      // log2 of the page size
  uint32_t page_stride;  // bytes from page to page of a layer
};

// A sequence's geometry, from device memory (every thread of a workgroup computes the same).
struct Seq {
  int slot, len, n, c0;     // n rows from c0 on
  int lo;                   // keys below lo are seen by no row but as sinks
  int n_sink, first, tiles; // key tiles: [0, n_sink), then first ..; `tiles` in all, at least one
  int col_tiles;            // tiles of C (row, head) columns of one key/value head; 0: not this kernel's
  bool ordered;             // its bounds are in order: the first starts at row 0, and c0 <= end <= rows
};

// A sequence whose bounds are out of order, and those after it, have no rows (the ones before it then
// share none): their rows are the rest that clear_rest clears.
__device__ __forceinline__ bool bounds_ok(const AttnArgs &g, int s, int c0, int c1) {
  return (s > 0 ? c0 >= 0 : c0 == 0) && c1 >= c0 && c1 <= g.a.b.rows;
}

template <int C>
__device__ Seq seq_of(const AttnArgs &g, int s, bool flag) {
  const trellis_kv4_batch &b = g.a.b;
  Seq q;
  const int c0 = ldg(b.cu + s), c1 = ldg(b.cu + s + 1);
  q.ordered = bounds_ok(g, s, c0, c1);
  q.c0 = q.ordered ? c0 : 0;
  q.n = q.ordered ? c1 - c0 : 0;
  q.slot = b.slots ? ldg(b.slots + s) : s;
  bool ok = (uint32_t)q.slot < (uint32_t)b.n_slots;
  q.slot = ok ? q.slot : 0;
  q.len = ldg(b.lens + q.slot);
  if (q.len < 0 || q.len > (long long)b.max_pages * g.a.c.page_size) ok = false;
  if (!ok) q.len = 0;
  if (flag && !(ok && q.ordered)) kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);
  const int lo = q.len - q.n - g.a.window + 1;  // of the first row
  q.lo = g.a.window && lo > 0 ? lo : 0;
  q.first = q.lo / kTile;
  const int sinks = (min(g.a.sinks, q.len) + kTile - 1) / kTile;
  q.n_sink = min(sinks, q.first);
  q.tiles = max(1, q.n_sink + (q.len + kTile - 1) / kTile - q.first);
  const long long cols = (long long)q.n * g.group;
  q.col_tiles = (cols <= g.few) == (C <= kCols) ? (int)((cols + C - 1) / C) : 0;
  return q;
}

// The same with every field in scalar registers, from lane `l`.
__device__ __forceinline__ Seq seq_from(const Seq &q, int l) {
  Seq r;
  r.slot = __builtin_amdgcn_readlane(q.slot, l);
  r.len = __builtin_amdgcn_readlane(q.len, l);
  r.n = __builtin_amdgcn_readlane(q.n, l);
  r.c0 = __builtin_amdgcn_readlane(q.c0, l);
  r.lo = __builtin_amdgcn_readlane(q.lo, l);
  r.n_sink = __builtin_amdgcn_readlane(q.n_sink, l);
  r.first = __builtin_amdgcn_readlane(q.first, l);
  r.tiles = __builtin_amdgcn_readlane(q.tiles, l);
  r.col_tiles = __builtin_amdgcn_readlane(q.col_tiles, l);
  return r;
}

__device__ __forceinline__ int tile_at(const Seq &q, int t) { return t < q.n_sink ? t : q.first + t - q.n_sink; }

// Exchanges between the lanes l, l ^ 32 (16) of two registers: afterwards a has both registers'
// lanes of the lower half (even rows of 16), b the upper.
__device__ __forceinline__ void swap32(float &a, float &b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  const uint32_t x = r[0], y = r[1];  // (a bit cast of a vector's element itself reads element 0)
  a = __builtin_bit_cast(float, x);
  b = __builtin_bit_cast(float, y);
}
__device__ __forceinline__ void swap16(float &a, float &b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  const uint32_t x = r[0], y = r[1];  // (a bit cast of a vector's element itself reads element 0)
  a = __builtin_bit_cast(float, x);
  b = __builtin_bit_cast(float, y);
}
// The value's maximum / sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max4(float v) {
  float a = v, b = v;
  swap16(a, b);
  a = b = fmaxf(a, b);
  swap32(a, b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float sum4(float v) {
  float a = v, b = v;
  swap16(a, b);
  a = b = a + b;
  swap32(a, b);
  return a + b;
}

__device__ __forceinline__ uint32_t max4u(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  const uint32_t x = a[0], y = a[1], w = x > y ? x : y;
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  const uint32_t s = b[0], t = b[1];
  return s > t ? s : t;
}

// Byte of a power of two 2^e as a matrix instruction's scale.
__device__ __forceinline__ constexpr int scale_byte(int e) { return 127 + e; }

// A column is a row and one of the key/value head's query heads.  Columns are counted from a uniform
// one, up to 63 on, so that only that one is divided.
struct ColumnBase {
  int row, head;
};
__device__ __forceinline__ ColumnBase column_base(const AttnArgs &g, int col0) {
  const int row = __builtin_amdgcn_readfirstlane(col0 / g.group);
  return {row, col0 - row * g.group};
}
__device__ __forceinline__ ColumnBase column_at(const AttnArgs &g, const ColumnBase &from, int i) {
  const uint32_t x = from.head + i, r = __umul24(x, g.per_group) >> 16;
  return {from.row + (int)r, (int)(x - __umul24(r, g.group))};
}

// Sixteen lanes to a column (the `col`-th from `from` on), eight elements each.
template <int NB>
struct QueryRaw {
  u32x4 x[NB];
};
template <int NB>
__device__ __forceinline__ QueryRaw<NB> load_query(const AttnArgs &g, const Seq &q, int head, const ColumnBase &from, int col) {
  QueryRaw<NB> r;
  const ColumnBase c = column_at(g, from, col);
  const bool ok = c.row < q.n;
  const uint16_t *p = static_cast<const uint16_t *>(g.a.q.p);
  if (ok) p += (int64_t)(q.c0 + c.row) * g.a.q.row_stride + (head * g.group + c.head) * g.a.q.head_stride + 8 * (threadIdx.x & 15);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    r.x[nb] = u32x4{0, 0, 0, 0};
    if (ok) r.x[nb] = ldg(reinterpret_cast<const u32x4 *>(p + nb * 128));
  }
  return r;
}

constexpr int kRowF = 132;  // floats of a column in shared memory: 128, and 4 to spread the banks

// Rotates column c of `to`, 16 lanes a column, times the softmax's scale and log2 e; even elements of each
// 32 first, as the conversion takes them.
template <bool BF, int NB>
__device__ __forceinline__ void stage_query(const AttnArgs &g, const QueryRaw<NB> &raw, int c, float (*to)[kCols][kRowF]) {
  const int i = threadIdx.x & 15, k = kv4_fwht16_place(i);
  const float factor = g.a.scale * (kLog2e * kRsqrt128) * kv4_fwht16_sign(i);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float x[8];
    kv4_unpack8<BF>(raw.x[nb], x);
    kv4_fwht16_signed(x, i);
    float *at = to[nb][c] + 32 * (k >> 2) + 4 * (k & 3);
    *reinterpret_cast<floatx4 *>(at) = floatx4{x[0], x[2], x[4], x[6]} * factor;
    *reinterpret_cast<floatx4 *>(at + 16) = floatx4{x[1], x[3], x[5], x[7]} * factor;
  }
}

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx32 __attribute__((ext_vector_type(32)));
typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));

// A block of a column as a matrix operand: lane (n, g) has elements 32 g .. 32 g + 31 of column n, as
// three E2M3 parts.  (Their products take half the time of E4M3's.  A part's steps are fixed where
// E4M3's shrink with the element, so three reach 2^-12 / 3.75 of the block's largest element, not of each;
// a score is a sum over the block, whose error the largest elements set either way.)
struct QueryBlock {
  u32x6 part[3];
  int scale;  // a byte a part: its power of two as the matrix instructions take it
  float add;  // NaN where the block is not finite: no E2M3 number says so
};

__device__ __forceinline__ QueryBlock take_block(const float *from) {
  const floatx4 *p = reinterpret_cast<const floatx4 *>(from);
  QueryBlock q;
  floatx16 x[2];  // elements 2 j, 2 j + 1
  uint32_t top = 0;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const floatx4 v = p[t];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float w = v[e];
      x[t >> 2][4 * (t & 3) + e] = w;
      // the largest magnitude as an integer: infinity is above every number, a NaN above infinity
      const uint32_t u = __builtin_bit_cast(uint32_t, w) & 0x7FFFFFFFu;
      top = u > top ? u : top;
    }
  }
  top = max4u(top);
  q.add = top >= 0x7F800000u ? __builtin_nanf("") : 0.f;
  // The largest comes to [3.75, 7.5), so nothing saturates; what a part leaves is at most 0.25, then
  // 0.125, in its units: the next one's are 16, then 32 times smaller.
  const int e = max((int)((top + 0x00100000u) >> 23), 24);
  q.scale = (e - 2) | (e - 6) << 8 | (e - 11) << 16;
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const float unit = __builtin_bit_cast(float, (uint32_t)(e - (s == 0 ? 2 : s == 1 ? 6 : 11)) << 23);
    q.part[s] = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(x[0], x[1], unit);
    if (s < 2) {
      const floatx32 back = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(q.part[s], unit);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[0][j] -= back[2 * j], x[1][j] -= back[2 * j + 1];
    }
  }
  return q;
}

__device__ __forceinline__ v8i read8(const int *p) {
  const v4i a = *reinterpret_cast<const v4i *>(p), b = *reinterpret_cast<const v4i *>(p + 4);
  return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Clears the rows from `end` on, where the n_seq sequences whose bounds are in order end (one workgroup).
template <int NB, int THREADS>
__device__ __forceinline__ void clear_rest(const AttnArgs &g, int n_seq, int end) {
  if (n_seq == g.a.b.n_seq && end == g.a.b.rows) return;
  if (threadIdx.x == 0) kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);
  const size_t words = (size_t)g.a.n_q_heads * 64 * NB;
  for (size_t i = end * words + threadIdx.x; i < g.a.b.rows * words; i += THREADS) static_cast<uint32_t *>(g.a.y)[i] = 0;
  if (g.a.lse)
    for (size_t i = (size_t)end * g.a.n_q_heads + threadIdx.x; i < (size_t)g.a.b.rows * g.a.n_q_heads; i += THREADS) g.a.lse[i] = kNegInf;
}

// Writes one column block's result: 16 lanes, eight elements each, still rotated and not
// normalised.
template <bool BF>
__device__ __forceinline__ void write_block(const AttnArgs &g, const Seq &q, int head, const ColumnBase &c, int nb, float (&v)[8],
                                            float m, float l) {
  const int i = threadIdx.x & 15;
  kv4_fwht16_signed(v, i);
  const float f = l == 0.f ? 0.f : kv4_fwht16_sign(i) * kRsqrt128 / l;  // (nothing seen: zero)
#pragma unroll
  for (int t = 0; t < 8; ++t) v[t] *= f;
  if (l == 0.f)
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = 0.f;
  const size_t at = (size_t)(q.c0 + c.row) * g.a.n_q_heads + head * g.group + c.head;
  uint16_t *y = static_cast<uint16_t *>(g.a.y) + at * g.a.c.head_dim + nb * 128 + 8 * kv4_fwht16_place(i);
  *reinterpret_cast<u32x4 *>(y) = kv4_pack8<BF>(v);
  if (g.a.lse && nb == 0 && i == 0) g.a.lse[at] = l == 0.f ? kNegInf : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Many columns per sequence (kv4_attn_wide.hip).
size_t kv4_attn_wide_parts(const trellis_kv4_cache &c, const trellis_kv4_batch &b, int n_q_heads);  // bytes of g.parts
hipError_t launch_kv4_attn_wide(const AttnArgs &g, hipStream_t stream);

}  // namespace trellis
