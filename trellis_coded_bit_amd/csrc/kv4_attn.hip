// Attention over the 4-bit key/value cache, on the scaled matrix instructions.
//
// Mathematics.  With q' = H q (rotated once per row) a score is q . k = sum over blocks of
// ks * (q' . kc): kc the stored E2M1 codes, ks the block's scale.  The codes are matrix operands
// as they lie in memory: v_mfma_scale_f32_16x16x128_f8f6f4 takes an E2M1 operand against an
// E4M3 one, 128 products deep, so a key is never unpacked and its scale is one multiplication
// per score.  Likewise y' = sum_j (p_j vs_j) vc_j with the value's scale taken into the weight,
// and y = H y' at the end.
//
// Precision.  What meets the codes is split into E4M3 parts, each the rounding of what the last
// one left: a query into three (within 2^-12 of each element, its own 16 bits for fp16), with one
// power of two per (row, block); a weight p_j vs_j into three (within 2^-12), with one power of
// two per tile of 128 keys.  Products and sums are fp32, as are the maxima, the sums of weights and
// everything that is joined.
#include "kv4_device.h"

namespace trellis {

namespace {

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
  float *parts;        // [workgroups][2][C][D + 8]: unnormalised sums, then maximum, sum of weights
  int group;           // query heads per key/value head
  int page_shift;      // log2 of the page size
  uint32_t page_stride;  // bytes from page to page of a layer
};

// A sequence's geometry, from device memory (every thread of a workgroup computes the same).
struct Seq {
  int slot, len, n, c0;     // n rows from c0 on
  int lo;                   // keys below lo are seen by no row but as sinks
  int n_sink, first, tiles; // key tiles: [0, n_sink), then first ..; `tiles` in all, at least one
  int col_tiles;            // tiles of C (row, head) columns of one key/value head
};

template <int C>
__device__ Seq seq_of(const AttnArgs &g, int s, bool flag) {
  const trellis_kv4_batch &b = g.a.b;
  Seq q;
  const int c0 = ldg(b.cu + s), c1 = ldg(b.cu + s + 1);
  const bool rows_ok = c0 >= 0 && c1 >= c0 && c1 <= b.rows;
  q.c0 = rows_ok ? c0 : 0;
  q.n = rows_ok ? c1 - c0 : 0;
  q.slot = b.slots ? ldg(b.slots + s) : s;
  bool ok = (uint32_t)q.slot < (uint32_t)b.n_slots;
  q.slot = ok ? q.slot : 0;
  q.len = ldg(b.lens + q.slot);
  if (q.len < 0 || q.len > (long long)b.max_pages * g.a.c.page_size) ok = false;
  if (!ok) q.len = 0;
  if (flag && !(ok && rows_ok)) kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);
  const int lo = q.len - q.n - g.a.window + 1;  // of the first row
  q.lo = g.a.window && lo > 0 ? lo : 0;
  q.first = q.lo / kTile;
  const int sinks = (min(g.a.sinks, q.len) + kTile - 1) / kTile;
  q.n_sink = min(sinks, q.first);
  q.tiles = max(1, q.n_sink + (q.len + kTile - 1) / kTile - q.first);
  q.col_tiles = (int)(((long long)q.n * g.group + C - 1) / C);
  return q;
}

__device__ __forceinline__ int tile_at(const Seq &q, int t) { return t < q.n_sink ? t : q.first + t - q.n_sink; }

// One wave's share of shared memory: a value tile (then, at a segment's end, its sums), and the
// tile's scales, reordered so that a lane's 32 keys are contiguous.
constexpr int kRowF = 132;  // floats of a column's sums: 128, and 4 to spread the banks
template <int NB, int R>
struct WaveLds {
  alignas(16) char v[NB * kCols * kRowF * 4];  // >= NB * 8 KiB
  alignas(16) uint16_t ks[NB][kTile], vs[NB][kTile];
  alignas(16) int w[R > 1 ? 4 * (kCols / R) * 3 + 1 : 1][8];  // weights' parts on their way between lanes; then zeros
};

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

// H_128 over 32 values a lane and the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ void fwht_cols(float (&x)[32]) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1)
#pragma unroll
    for (int t = 0; t < 32; ++t)
      if ((t & h) == 0) {
        const float a = x[t], b = x[t + h];
        x[t] = a + b;
        x[t + h] = a - b;
      }
#pragma unroll
  for (int t = 0; t < 32; t += 2) {
    float a = x[t], b = x[t + 1];
    swap16(a, b);
    float s = a + b, d = a - b;
    swap16(s, d);
    swap32(s, d);
    a = s + d;
    b = s - d;
    swap32(a, b);
    x[t] = a;
    x[t + 1] = b;
  }
}

// Byte of a power of two 2^e as a matrix instruction's scale.
__device__ __forceinline__ constexpr int scale_byte(int e) { return 127 + e; }

// 16 columns' rotated queries as matrix operands.  Lane (n = l & 15, g = l >> 4) holds column
// n's elements 16 g .. + 15 and 64 + 16 g .. + 15 of a block: the E4M3 operand's order.
template <int NB>
struct Queries {
  v8i part[NB][3];
  float cf[NB];  // score = cf * (sum over parts), in powers of two; >= 0
  int pos;       // the column's position (-1: sees nothing)
};

template <bool BF, int NB, int R>
__device__ __forceinline__ Queries<NB> load_queries(const AttnArgs &g, const Seq &q, int head, int col0) {
  Queries<NB> r;
  const int lane = threadIdx.x & 63, c = col0 + (lane & (kCols / R - 1)), k = lane >> 4;
  const bool ok = c < (long long)q.n * g.group;
  const int i = ok ? c / g.group : 0, h = head * g.group + (ok ? c % g.group : 0);
  r.pos = ok ? q.len - q.n + i : -1;
  const uint16_t *p = static_cast<const uint16_t *>(g.a.q.p) + (int64_t)(q.c0 + i) * g.a.q.row_stride + h * g.a.q.head_stride;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float x[32];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      u32x4 raw = {0, 0, 0, 0};
      if (ok) raw = ldg(reinterpret_cast<const u32x4 *>(p + nb * 128 + (w >> 1) * 64 + 16 * k + (w & 1) * 8));
      float v[8];
      kv4_unpack8<BF>(raw, v);
#pragma unroll
      for (int t = 0; t < 8; ++t) x[8 * w + t] = v[t];
    }
    fwht_cols(x);
    float top = 0.f;
    bool finite = true;
#pragma unroll
    for (int t = 0; t < 32; ++t) {
      top = fmaxf(top, fabsf(x[t]));
      finite &= fabsf(x[t]) <= 3.4028234e38f;
    }
    top = max4(finite ? top : __builtin_inff());
    // the largest element comes to [128, 256); a column that is not finite becomes NaN
    const int e = max((int)(__builtin_bit_cast(uint32_t, top) >> 23), 8);
    float f = __builtin_bit_cast(float, (uint32_t)min(261 - e, 254) << 23);
    if (top > 3.4028234e38f) f = __builtin_nanf("");
    if (g.a.scale < 0.f) f = -f;
    r.cf[nb] = __builtin_bit_cast(float, (uint32_t)(e - 7) << 23) * (fabsf(g.a.scale) * kLog2e * kRsqrt128);
#pragma unroll
    for (int t = 0; t < 32; ++t) x[t] *= f;
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        int o = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * w], x[4 * w + 1], 0, false);
        o = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * w + 2], x[4 * w + 3], o, true);
        r.part[nb][s][w] = o;
        if (s < 2) {  // what is left, times 16: at most 128
          const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(o, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(o, true);
          x[4 * w] = (x[4 * w] - lo[0]) * 16.f;
          x[4 * w + 1] = (x[4 * w + 1] - lo[1]) * 16.f;
          x[4 * w + 2] = (x[4 * w + 2] - hi[0]) * 16.f;
          x[4 * w + 3] = (x[4 * w + 3] - hi[1]) * 16.f;
        }
      }
  }
  return r;
}

// A tile's codes and scales in registers: a wave's 16-byte loads, lane l the key l & 15 of a
// subtile of 16 and the elements 32 (l >> 4) .. + 31 (keys: the E2M1 operand's order), or the
// token l >> 2 and its 16-byte part l & 3 (values, bound for shared memory).
template <int NB>
struct Tile {
  v4i k[NB][8], v[NB][8];
  uint32_t ks[NB], vs[NB];  // scales of the tokens 2 l, 2 l + 1
  int page;                 // of these tokens
};

// The pages of a tile: lane l has that of its tokens 2 l, 2 l + 1, or -1 where there is none:
// past the length, or a number that is no page.
__device__ __forceinline__ int tile_pages(const AttnArgs &g, const Seq &q, int tile) {
  const int tok = tile * kTile + 16 * ((threadIdx.x & 63) >> 3);
  if (tok >= q.len) return -1;
  const int page = ldg(g.a.b.table + (size_t)q.slot * g.a.b.max_pages + (tok >> g.page_shift));
  if ((uint32_t)page < (uint32_t)g.a.c.n_pages) return page;
  if (tok + 15 >= q.lo || tok < g.a.sinks) kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);  // some row would see it
  return -1;
}

// `base`: the head's chunk of page 0 of the layer.  (A subtile without a page reads page 0's.)
template <int NB>
__device__ __forceinline__ void load_tile(const AttnArgs &g, const char *base, int tile, int page, Tile<NB> &x) {
  const uint32_t lane = threadIdx.x & 63, T = g.a.c.page_size;
  const uint32_t lk = (lane & 15) * 64 + (lane >> 4) * 16, lv = lane * 16 + NB * T * 64;
  const uint64_t mine = (uint64_t)(uint32_t)max(page, 0) * g.page_stride;
  x.page = page;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)mine, 8 * j), hi = __builtin_amdgcn_readlane((uint32_t)(mine >> 32), 8 * j);
    const char *p = base + (((uint64_t)hi << 32) | lo) + ((tile * kTile + 16 * j) & (T - 1)) * 64;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      x.k[nb][j] = ldg(reinterpret_cast<const v4i *>(p + nb * T * 64 + lk));
      x.v[nb][j] = ldg(reinterpret_cast<const v4i *>(p + nb * T * 64 + lv));
    }
  }
  const char *p = base + mine + 128 * NB * T + ((tile * kTile + 2 * lane) & (T - 1)) * 2;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    x.ks[nb] = ldg(reinterpret_cast<const uint32_t *>(p + nb * T * 2));
    x.vs[nb] = ldg(reinterpret_cast<const uint32_t *>(p + (NB + nb) * T * 2));
  }
}

// Moves a tile's values and scales to the wave's shared memory.  Keys that no row sees get
// scale zero.  The value scales are multiplied by a power of two that brings the tile's largest
// to [128, 256); returns its inverse as a matrix instruction's scale byte, per block.
// A token's four 16-byte parts are permuted by its subtile, which spreads the transposed reads
// below over the banks.
template <int NB, int R>
__device__ __forceinline__ void stage_tile(const AttnArgs &g, const Seq &q, int tile, const Tile<NB> &x, WaveLds<NB, R> &lds,
                                           int (&vbyte)[NB]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<v4i *>(lds.v + nb * 8192 + j * 1024 + (lane >> 2) * 64 + (((lane & 3) ^ (j & 3)) * 16)) = x.v[nb][j];
  const int tok = tile * kTile + 2 * lane;
  const bool here = x.page >= 0;
  const uint32_t keep = (here && tok < q.len && (tok >= q.lo || tok < g.a.sinks) ? 0xFFFFu : 0u) |
                        (here && tok + 1 < q.len && (tok + 1 >= q.lo || tok + 1 < g.a.sinks) ? 0xFFFF0000u : 0u);
  const int at = ((lane & 7) >> 1) * 32 + (lane >> 3) * 4 + 2 * (lane & 1);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    *reinterpret_cast<uint32_t *>(&lds.ks[nb][at]) = x.ks[nb] & keep;
    const uint32_t w = x.vs[nb] & keep;
    const float a = __builtin_bit_cast(float, w << 16), b = __builtin_bit_cast(float, w & 0xFFFF0000u);
    // (a NaN scale stands for a NaN value; it does not set the power of two)
    float top = fmaxf(fabsf(a) <= 3.4028234e38f ? fabsf(a) : 0.f, fabsf(b) <= 3.4028234e38f ? fabsf(b) : 0.f);
    top = fmaxf(top, lane_xor<1>(top));
    top = fmaxf(top, lane_xor<2>(top));
    top = fmaxf(top, lane_xor<4>(top));
    top = fmaxf(top, lane_xor<8>(top));
    top = max4(top);
    const int e = __builtin_amdgcn_readfirstlane(max((int)(__builtin_bit_cast(uint32_t, top) >> 23), 32));
    const float f = __builtin_bit_cast(float, (uint32_t)(261 - e) << 23);
    const uint32_t fa = __builtin_bit_cast(uint32_t, a * f), fb = __builtin_bit_cast(uint32_t, b * f);
    *reinterpret_cast<uint32_t *>(&lds.vs[nb][at]) = (fa >> 16) | (fb & 0xFFFF0000u);
    vbyte[nb] = e - 7;
  }
}

// A lane's own keys.  With R = 16 / C columns held R times over (few columns: the matrix
// instruction is 16 wide anyway), replica r of a column takes the NT = 8 / R subtiles from r NT
// on through the softmax.  Their scales: 2 NT words from shared memory.
template <int R>
__device__ __forceinline__ void read_scales(const uint16_t *s, uint32_t (&w)[16 / R]) {
  const int lane = threadIdx.x & 63, r = (lane & 15) / (kCols / R);
  const u32x4 *p = reinterpret_cast<const u32x4 *>(s + (lane >> 4) * 32 + r * (32 / R));
#pragma unroll
  for (int t = 0; t < 4 / R; ++t) {
    const u32x4 v = p[t];
    w[4 * t] = v[0], w[4 * t + 1] = v[1], w[4 * t + 2] = v[2], w[4 * t + 3] = v[3];
  }
}
template <int N>
__device__ __forceinline__ float scale_of(const uint32_t (&w)[N], int t, int i) {
  const uint32_t x = w[2 * t + (i >> 1)];
  return __builtin_bit_cast(float, (i & 1) ? x & 0xFFFF0000u : x << 16);
}

// 16 columns' running sums.  Lane (n, g): column n; elements 16 dt + 4 g + i of o[nb][dt][i].  With
// R > 1 the replicas of a column hold the sums over the weights' parts (R = 4: one part each;
// R = 2: the first and third, and the second); they are added at the end.
template <int NB>
struct Sums {
  floatx4 o[NB][8];
  float m;  // maximum so far, in powers of two, the same in the column's four lanes
  float l;  // this lane's share of the sum of weights
};

// A tile's values as the left operand of the second product: rows are elements 16 dt + (l & 15),
// the 32 keys of the lane's depth share those that the weights' E4M3 operand has there (lane
// group g of it: keys 16 t + 4 g + i, t = 0..3 in its first half, 4..7 in its second).
template <int NB, int R>
__device__ __forceinline__ v8i read_values(const WaveLds<NB, R> &lds, int nb, int dt) {
  const int lane = threadIdx.x & 63, gv = lane >> 4, r = lane & 15;
  const int tok = 64 * (gv >> 1) + 16 * (r >> 2) + 8 * (gv & 1) + (r & 3);
  const char *p = lds.v + nb * 8192 + tok * 64 + (((dt >> 1) ^ (r >> 2)) * 16) + (dt & 1) * 8;
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  const v2i a = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_v2i *)p);
  const v2i b = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_v2i *)(p + 4 * 64));
  return v8i{a[0], a[1], b[0], b[1], 0, 0, 0, 0};
}

// Scores of a lane's own keys: x[t][i] belongs to key 16 (r NT + t) + 4 g + i and the lane's
// column, in units of cf[0] (one block) or in powers of two (two blocks).
template <int NB, int R>
__device__ __forceinline__ void scores(const v4i (&k)[NB][8], const Queries<NB> &qr, const WaveLds<NB, R> &lds,
                                       float (&x)[8 / R][4]) {
  constexpr int NT = 8 / R;
  const int r = (threadIdx.x & 15) / (kCols / R);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    uint32_t ks[16 / R];
    read_scales<R>(lds.ks[nb], ks);
    float y[NT][4];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const v8i a = {k[nb][t][0], k[nb][t][1], k[nb][t][2], k[nb][t][3], 0, 0, 0, 0};
      floatx4 s = {0.f, 0.f, 0.f, 0.f};
      s = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, qr.part[nb][0], s, 4, 0, 0, scale_byte(0), 0, scale_byte(0));
      s = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, qr.part[nb][1], s, 4, 0, 0, scale_byte(0), 0, scale_byte(-4));
      s = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, qr.part[nb][2], s, 4, 0, 0, scale_byte(0), 0, scale_byte(-8));
#pragma unroll
      for (int i = 0; i < 4; ++i) y[t % NT][i] = t < NT || r == t / NT ? s[i] : y[t % NT][i];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float z = y[t][i] * scale_of(ks, t, i);
        if (NB == 1) x[t][i] = z;
        else x[t][i] = nb ? fmaf(z, qr.cf[nb], x[t][i]) : z * qr.cf[nb];
      }
  }
}

// Four weights as three E4M3 parts, one word each: what is left is brought up 32 times before the
// next rounding (at most 256).
__device__ __forceinline__ void split3(const float (&w)[4], int &p0, int &p1, int &p2) {
  int o = __builtin_amdgcn_cvt_pk_fp8_f32(w[0], w[1], 0, false);
  o = __builtin_amdgcn_cvt_pk_fp8_f32(w[2], w[3], o, true);
  floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8(o, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(o, true);
  const float x0 = w[0] - a[0], x1 = w[1] - a[1], x2 = w[2] - b[0], x3 = w[3] - b[1];
  p0 = o;
  constexpr float k1 = 1.f / 32, k2 = 1.f / 1024;
  v2s z = {0, 0};
  z = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(z, x0, x1, k1, false);
  z = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(z, x2, x3, k1, true);
  p1 = __builtin_bit_cast(int, z);
  a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(p1, k1, false);
  b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(p1, k1, true);
  z = v2s{0, 0};
  z = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(z, x0 - a[0], x1 - a[1], k2, false);
  z = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(z, x2 - b[0], x3 - b[1], k2, true);
  p2 = __builtin_bit_cast(int, z);
}

__device__ __forceinline__ v8i read8(const int *p) {
  const v4i a = *reinterpret_cast<const v4i *>(p), b = *reinterpret_cast<const v4i *>(p + 4);
  return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// One tile into a column tile's sums.  MASK: some row does not see some key of the tile; bad: bit
// 8 t of a subtile t without a page.
template <int NB, int R, bool MASK>
__device__ __forceinline__ void add_tile(const AttnArgs &g, int tile, uint64_t bad, const int (&vbyte)[NB],
                                         float (&x)[8 / R][4], const Queries<NB> &qr, WaveLds<NB, R> &lds, Sums<NB> &sum) {
  constexpr int NT = 8 / R, C = kCols / R;
  const int lane = threadIdx.x & 63, r = (lane & 15) / C, k = lane >> 4;
  uint32_t seen = 0;
  if (MASK) {
    const int k0 = tile * kTile + 16 * NT * r + 4 * k, rel = qr.pos - k0;
    const int after = g.a.window ? rel - g.a.window : -0x40000000, sink = g.a.window ? g.a.sinks - k0 : 0;
    const uint64_t mine = bad >> (8 * NT * r);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 16 * t + i;
        const bool ok = j <= rel && (j > after || j < sink) && !((mine >> (8 * t)) & 1);
        x[t][i] = ok ? x[t][i] : kNegInf;
        seen |= ok ? 1u << (4 * t + i) : 0u;
      }
  }
  float top = kNegInf;
#pragma unroll
  for (int t = 0; t < NT; ++t) top = fmaxf(fmaxf(fmaxf(top, x[t][0]), fmaxf(x[t][1], x[t][2])), x[t][3]);
  if (R >= 4) top = fmaxf(top, lane_xor<4>(top));
  if (R >= 2) top = fmaxf(top, lane_xor<8>(top));
  top = max4(top);
  const float cf = NB == 1 ? qr.cf[0] : 1.f;
  const float m = fmaxf(sum.m, top == kNegInf ? kNegInf : top * cf);
  const float mu = m == kNegInf ? 0.f : m;  // nothing seen so far
  const float alpha = __builtin_amdgcn_exp2f(sum.m - mu);
  sum.m = m;
  float add = 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (cf may be zero, and a score that is not seen minus infinity)
      const float d = MASK && !((seen >> (4 * t + i)) & 1) ? kNegInf : fmaf(x[t][i], cf, -mu);
      x[t][i] = __builtin_amdgcn_exp2f(d);
      add += x[t][i];
    }
  sum.l = fmaf(sum.l, alpha, add);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    uint32_t vs[16 / R];
    read_scales<R>(lds.vs[nb], vs);
    int part[3][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = x[t][i] * scale_of(vs, t, i);
        if (MASK && !((seen >> (4 * t + i)) & 1)) w[i] = 0.f;  // (its scale may be NaN)
      }
      split3(w, part[0][t], part[1][t], part[2][t]);
    }
    v8i p0, p1, p2;
    if constexpr (R == 1) {
#pragma unroll
      for (int t = 0; t < 8; ++t) p0[t] = part[0][t], p1[t] = part[1][t], p2[t] = part[2][t];
    } else {
      // replica r turns from the keys r NT .. of all parts to all keys of part r
      const int h = lane & (C - 1), row = (k * C + h) * 3;
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        int *to = lds.w[row + s] + r * NT;
        if constexpr (R == 4) *reinterpret_cast<v2i *>(to) = v2i{part[s][0], part[s][1]};
        else *reinterpret_cast<v4i *>(to) = v4i{part[s][0], part[s][1], part[s][2], part[s][3]};
      }
      constexpr int zeros = 4 * C * 3;
      p0 = read8(lds.w[r < 3 ? row + r : zeros]);
      if constexpr (R == 2) p1 = read8(lds.w[r == 0 ? row + 2 : zeros]);
    }
    const int b0 = vbyte[nb] - (R > 1 ? 5 * r : 0);
#pragma unroll
    for (int dt = 0; dt < 8; ++dt) {
      const v8i v = read_values(lds, nb, dt);
      floatx4 o = sum.o[nb][dt] * alpha;
      o = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, p0, o, 4, 0, 0, scale_byte(0), 0, b0);
      if constexpr (R == 2) o = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, p1, o, 4, 0, 0, scale_byte(0), 0, vbyte[nb] - 10);
      if constexpr (R == 1) {
        o = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, p1, o, 4, 0, 0, scale_byte(0), 0, vbyte[nb] - 5);
        o = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, p2, o, 4, 0, 0, scale_byte(0), 0, vbyte[nb] - 10);
      }
      sum.o[nb][dt] = o;
    }
  }
}

// Writes one column block's result: 16 lanes, eight elements each, still rotated and not
// normalised.
template <bool BF>
__device__ __forceinline__ void write_block(const AttnArgs &g, const Seq &q, int head, int c, int nb, float (&v)[8], float m,
                                            float l) {
  const int i = threadIdx.x & 15;
  kv4_fwht16(v, threadIdx.x & 63);
  const float f = l == 0.f ? 0.f : kRsqrt128 / l;  // (nothing seen: zero)
#pragma unroll
  for (int t = 0; t < 8; ++t) v[t] *= f;
  if (l == 0.f)
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = 0.f;
  const size_t at = (size_t)(q.c0 + c / g.group) * g.a.n_q_heads + head * g.group + c % g.group;
  uint16_t *y = static_cast<uint16_t *>(g.a.y) + at * g.a.c.head_dim + nb * 128 + 8 * i;
  *reinterpret_cast<u32x4 *>(y) = kv4_pack8<BF>(v);
  if (g.a.lse && nb == 0 && i == 0) g.a.lse[at] = l == 0.f ? kNegInf : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Few columns per sequence: single and drafted tokens.  HBM (or, for short contexts, latency)
// bounds it: every key and value is read once and used for at most 16 columns.
//
// All sequences' (head, column tile, key tile) units stand in one line; each workgroup takes an
// equal stretch of it, whatever the lengths, and its four waves take the stretch's key tiles in
// turn, each with its own sums, joined in shared memory at a segment's end (a segment: one
// (sequence, head, column tile)).  A segment that several workgroups share is joined by the last
// of them to arrive, in order, so results do not depend on timing.
constexpr int kWaves = 4;
constexpr int kMinChunk = 8;  // tiles: two a wave; a join costs more than a second tile

template <int NB, int R>
struct NarrowLds {
  WaveLds<NB, R> wave[kWaves];
  float ml[kWaves][2][kCols];
  long long scan[kWaves + 1];
  long long found[2];
  int last;
};

// Exclusive prefix sum over the workgroup; *total gets the sum.
__device__ __forceinline__ long long prefix256(long long v, long long *lds, long long *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  long long x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long long y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  long long before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += lds[w];
    sum += lds[w];
  }
  *total = sum;
  return before + x - v;
}

__device__ __forceinline__ int padded(int tiles) { return (tiles + kMinChunk - 1) / kMinChunk * kMinChunk; }

template <bool BF, int NB, int R>
__global__ __launch_bounds__(256, NB == 1 ? 2 : 1) void kv4_attn_narrow_kernel(AttnArgs g) {
  constexpr int D = 128 * NB, C = kCols / R, kPart = C * (D + 8);
  extern __shared__ __attribute__((aligned(16))) char raw[];
  NarrowLds<NB, R> &lds = *reinterpret_cast<NarrowLds<NB, R> *>(raw);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n_seq = g.a.b.n_seq, Hk = g.a.c.n_kv_heads;
  // the line's length, with and without segments rounded up to whole chunks
  long long exact = 0, round = 0, w_exact = 0, w_round = 0, p_exact = 0, p_round = 0;
  for (int s0 = 0; s0 < n_seq; s0 += 256) {
    const int s = s0 + tid;
    w_exact = w_round = 0;
    if (s < n_seq) {
      const Seq q = seq_of<C>(g, s, blockIdx.x == 0);
      w_exact = (long long)Hk * q.col_tiles * q.tiles;
      w_round = (long long)Hk * q.col_tiles * padded(q.tiles);
    }
    long long t;
    p_exact = exact + prefix256(w_exact, lds.scan, &t);
    exact += t;
    p_round = round + prefix256(w_round, lds.scan, &t);
    round += t;
  }
  if (blockIdx.x == 0) {  // rows that no sequence has
    const int end = min(max(n_seq ? ldg(g.a.b.cu + n_seq) : 0, 0), g.a.b.rows);
    if (end < g.a.b.rows) {
      if (tid == 0) kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);
      const size_t words = (size_t)g.a.n_q_heads * D / 2;
      for (size_t i = end * words + tid; i < g.a.b.rows * words; i += 256) static_cast<uint32_t *>(g.a.y)[i] = 0;
      if (g.a.lse)
        for (size_t i = (size_t)end * g.a.n_q_heads + tid; i < (size_t)g.a.b.rows * g.a.n_q_heads; i += 256) g.a.lse[i] = kNegInf;
    }
  }
  const int G = gridDim.x;
  const bool whole = round <= (long long)kMinChunk * G;  // short contexts: whole chunks to a segment
  const long long U = whole ? round : exact, chunk = whole ? kMinChunk : (exact + G - 1) / G;
  long long u = blockIdx.x * chunk;
  const long long u1 = min(u + chunk, U);
  if (u >= u1) return;
  // the sequence of the first unit
  if (tid == 0) lds.found[0] = -1;
  __syncthreads();
  if (n_seq <= 256) {
    const long long p = whole ? p_round : p_exact, w = whole ? w_round : w_exact;
    if (u >= p && u < p + w) lds.found[0] = tid, lds.found[1] = p;
  } else {
    long long base = 0;
    for (int s0 = 0; s0 < n_seq; s0 += 256) {
      const int s = s0 + tid;
      long long w = 0, t;
      if (s < n_seq) {
        const Seq q = seq_of<C>(g, s, false);
        w = (long long)Hk * q.col_tiles * (whole ? padded(q.tiles) : q.tiles);
      }
      const long long p = base + prefix256(w, lds.scan, &t);
      if (u >= p && u < p + w) lds.found[0] = s, lds.found[1] = p;
      base += t;
      if (u < base) break;  // (uniform)
    }
  }
  __syncthreads();
  int s = __builtin_amdgcn_readfirstlane((int)lds.found[0]);
  if (s < 0) return;  // (the lengths changed under the call)
  long long pre = lds.found[1];
  Seq q = seq_of<C>(g, s, false);
  if (q.col_tiles == 0) return;
  for (;;) {
    const int per = whole ? padded(q.tiles) : q.tiles;
    const long long r = u - pre;
    const int seg = (int)(r / per), t0 = (int)(r % per);
    const int t1 = (int)min((long long)q.tiles, t0 + (u1 - u));
    const int head = seg / q.col_tiles, col0 = (seg % q.col_tiles) * C;
    const long long begin = pre + (long long)seg * per;
    // ---- this wave's tiles
    const Queries<NB> qr = load_queries<BF, NB, R>(g, q, head, col0);
    const int cols = (int)min((long long)C, (long long)q.n * g.group - col0);
    const int pos0 = q.len - q.n + col0 / g.group, pos1 = q.len - q.n + (col0 + cols - 1) / g.group;
    Sums<NB> sum;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) sum.o[nb][dt] = floatx4{0.f, 0.f, 0.f, 0.f};
    sum.m = kNegInf;
    sum.l = 0.f;
    WaveLds<NB, R> &mine = lds.wave[wave];
    if (R > 1 && lane < 8) mine.w[4 * C * 3][lane] = 0;
    const char *base = kv4_chunk(g.a.c, g.a.layer, 0, head);
    int t = t0 + wave;
    Tile<NB> x;
    int pages = -1;
    if (t < t1 && q.len > 0) {
      load_tile(g, base, tile_at(q, t), tile_pages(g, q, tile_at(q, t)), x);
      if (t + kWaves < t1) pages = tile_pages(g, q, tile_at(q, t + kWaves));
      while (true) {
        const int tile = tile_at(q, t), k0 = tile * kTile;
        const uint64_t bad = __ballot(x.page < 0);
        int vbyte[NB];
        stage_tile(g, q, tile, x, mine, vbyte);
        float sc[8 / R][4];
        scores<NB, R>(x.k, qr, mine, sc);
        const int next = t + kWaves;
        if (next < t1) {
          load_tile(g, base, tile_at(q, next), pages, x);
          if (next + kWaves < t1) pages = tile_pages(g, q, tile_at(q, next + kWaves));
        }
        const bool all = k0 + kTile - 1 <= pos0 && bad == 0 &&
                         (g.a.window == 0 || k0 > pos1 - g.a.window || k0 + kTile <= g.a.sinks);
        if (all) add_tile<NB, R, false>(g, tile, bad, vbyte, sc, qr, mine, sum);
        else add_tile<NB, R, true>(g, tile, bad, vbyte, sc, qr, mine, sum);
        if (next >= t1) break;
        t = next;
      }
    }
    // ---- join the waves
    float l = sum.l;
    if (R >= 4) l += lane_xor<4>(l);
    if (R >= 2) l += lane_xor<8>(l);
    l = sum4(l);
    if (lane < C) {
      lds.ml[wave][0][lane] = sum.m;
      lds.ml[wave][1][lane] = l;
    }
    float *own = reinterpret_cast<float *>(mine.v);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int dt = 0; dt < 8; ++dt)
        *reinterpret_cast<floatx4 *>(own + (nb * kCols + (lane & 15)) * kRowF + 16 * dt + 4 * (lane >> 4)) = sum.o[nb][dt];
    __syncthreads();
    const int col = (tid >> 4) % C, i = tid & 15;  // (with C < 16 the same by several threads)
    float M = kNegInf, L = 0.f, f[kWaves], v[NB][8];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) M = fmaxf(M, lds.ml[w][0][col]);
    const float mu = M == kNegInf ? 0.f : M;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      f[w] = __builtin_amdgcn_exp2f(lds.ml[w][0][col] - mu);
      L = fmaf(f[w], lds.ml[w][1][col], L);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[nb][e] = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float *o = reinterpret_cast<const float *>(lds.wave[w].v) + (nb * kCols + col) * kRowF + 8 * i;
        floatx4 a = *reinterpret_cast<const floatx4 *>(o), b = *reinterpret_cast<const floatx4 *>(o + 4);
#pragma unroll
        for (int r = 1; r < (R < 3 ? R : 3); ++r) {  // the weights' other parts
          a += *reinterpret_cast<const floatx4 *>(o + r * C * kRowF);
          b += *reinterpret_cast<const floatx4 *>(o + r * C * kRowF + 4);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[nb][e] = fmaf(f[w], a[e], v[nb][e]);
          v[nb][e + 4] = fmaf(f[w], b[e], v[nb][e + 4]);
        }
      }
    }
    const int w0 = (int)(begin / chunk), w1 = (int)((begin + q.tiles - 1) / chunk);  // the workgroups that share the segment
    if (w0 == w1) {
      if ((tid >> 4) < cols)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) write_block<BF>(g, q, head, col0 + col, nb, v[nb], M, L);
    } else {
      // ---- this workgroup's part, then the join by whoever arrives last
      const long long region = (long long)gridDim.x * 2 * kPart * 4;
      const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(g.parts, region);
      if ((tid >> 4) < cols) {
        const int at = (((int)blockIdx.x * 2 + ((int)blockIdx.x == w0 ? 1 : 0)) * kPart + col * (D + 8)) * 4;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const u32x4 a = {__builtin_bit_cast(uint32_t, v[nb][0]), __builtin_bit_cast(uint32_t, v[nb][1]),
                           __builtin_bit_cast(uint32_t, v[nb][2]), __builtin_bit_cast(uint32_t, v[nb][3])};
          const u32x4 b = {__builtin_bit_cast(uint32_t, v[nb][4]), __builtin_bit_cast(uint32_t, v[nb][5]),
                           __builtin_bit_cast(uint32_t, v[nb][6]), __builtin_bit_cast(uint32_t, v[nb][7])};
          __builtin_amdgcn_raw_buffer_store_b128(a, rs, at + (nb * 128 + 8 * i) * 4, 0, kSC1);
          __builtin_amdgcn_raw_buffer_store_b128(b, rs, at + (nb * 128 + 8 * i + 4) * 4, 0, kSC1);
        }
        if (i == 0) {
          const u32x2 ml = {__builtin_bit_cast(uint32_t, M), __builtin_bit_cast(uint32_t, L)};
          __builtin_amdgcn_raw_buffer_store_b64(ml, rs, at + D * 4, 0, kSC1);
        }
      }
      // every thread's stores have completed before the counter moves
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
      __syncthreads();
      if (tid == 0) {
        const uint32_t old = __hip_atomic_fetch_add(g.counters + w0, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        lds.last = old == (uint32_t)(w1 - w0);
        if (lds.last) __hip_atomic_store(g.counters + w0, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      if (__builtin_amdgcn_readfirstlane(lds.last)) {
        // `sub` shares of the parts run side by side where there are few columns
        const int width = cols <= 1 ? 1 : cols <= 2 ? 2 : cols <= 4 ? 4 : cols <= 8 ? 8 : 16, subs = kCols / width;
        const int sub = (tid >> 4) / width, c = (tid >> 4) % width;
        float m = kNegInf, l2 = 0.f, acc[NB][8];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[nb][e] = 0.f;
        if (c < cols)
#pragma unroll 4
          for (int w = w0 + sub; w <= w1; w += subs) {
            const int at = ((w * 2 + (w == w0 ? 1 : 0)) * kPart + c * (D + 8)) * 4;
            const u32x2 ml = __builtin_amdgcn_raw_buffer_load_b64(rs, at + D * 4, 0, kSC1);
            u32x4 p[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              p[nb][0] = __builtin_amdgcn_raw_buffer_load_b128(rs, at + (nb * 128 + 8 * i) * 4, 0, kSC1);
              p[nb][1] = __builtin_amdgcn_raw_buffer_load_b128(rs, at + (nb * 128 + 8 * i + 4) * 4, 0, kSC1);
            }
            const uint32_t mw = ml[0], lw = ml[1];
            const float pm = __builtin_bit_cast(float, mw), pl = __builtin_bit_cast(float, lw);
            const float m2 = fmaxf(m, pm), u2 = m2 == kNegInf ? 0.f : m2;
            const float fa = __builtin_amdgcn_exp2f(m - u2), fb = __builtin_amdgcn_exp2f(pm - u2);
            m = m2;
            l2 = l2 * fa + pl * fb;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                acc[nb][e] = acc[nb][e] * fa + __builtin_bit_cast(float, (uint32_t)p[nb][e >> 2][e & 3]) * fb;
          }
        // the shares, in order
        float *all = reinterpret_cast<float *>(lds.wave);
        float *put = all + tid * (8 * NB + 2);
        if (sub > 0) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 8; ++e) put[nb * 8 + e] = acc[nb][e];
          put[8 * NB] = m;
          put[8 * NB + 1] = l2;
        }
        __syncthreads();
        if (sub == 0 && c < cols) {
          for (int k = 1; k < subs; ++k) {
            const float *from = all + (tid + k * width * 16) * (8 * NB + 2);
            const float pm = from[8 * NB], m2 = fmaxf(m, pm), u2 = m2 == kNegInf ? 0.f : m2;
            const float fa = __builtin_amdgcn_exp2f(m - u2), fb = __builtin_amdgcn_exp2f(pm - u2);
            m = m2;
            l2 = l2 * fa + from[8 * NB + 1] * fb;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[nb][e] = acc[nb][e] * fa + from[nb * 8 + e] * fb;
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) write_block<BF>(g, q, head, col0 + c, nb, acc[nb], m, l2);
        }
      }
    }
    // ---- the next segment
    u = min(u1, begin + per);
    if (u >= u1) break;
    __syncthreads();  // shared memory is free again
    while (u >= pre + (long long)Hk * q.col_tiles * per) {
      pre += (long long)Hk * q.col_tiles * (whole ? padded(q.tiles) : q.tiles);
      if (++s >= n_seq) return;  // (as above)
      q = seq_of<C>(g, s, false);
      if (q.col_tiles > 0) break;
    }
  }
}

// How often the narrow kernel holds a column: as many columns as the sequences' rows are known or
// expected to have, up to 4, 8 or 16 a tile.  64 ragged contexts of 32 / 8 heads (4 columns):
// MEASURED_R.
int replicas(const trellis_kv4_cache &c, const trellis_kv4_batch &b, int n_q_heads, int max_rows) {
  const long long rows = max_rows > 0 ? max_rows : ((long long)b.rows + b.n_seq - 1) / b.n_seq;
  const long long cols = rows * (n_q_heads / c.n_kv_heads);
  return cols <= 4 ? 4 : cols <= 8 ? 2 : 1;
}

// Workgroups of the narrow kernel: as many as are resident at once, and no more than the
// capacity of the tables can use.
int narrow_grid(const trellis_kv4_cache &c, const trellis_kv4_batch &b, int n_q_heads, int C) {
  const long long group = n_q_heads / c.n_kv_heads;
  const long long tiles = ((long long)b.max_pages * c.page_size + kTile - 1) / kTile;
  const long long cols = ((long long)b.rows * group + C - 1) / C + b.n_seq;  // column tiles, at most
  const long long chunks = (tiles + kMinChunk - 1) / kMinChunk;
  const long long most = (long long)micro_cus() * (c.head_dim == 128 ? 2 : 1);
  const double want = (double)cols * c.n_kv_heads * chunks;
  return want < (double)most ? (want < 1 ? 1 : (int)want) : (int)most;
}

template <bool BF, int NB, int R>
hipError_t launch_narrow(const AttnArgs &g, hipStream_t stream) {
  const size_t lds = sizeof(NarrowLds<NB, R>);
  const auto kernel = kv4_attn_narrow_kernel<BF, NB, R>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<narrow_grid(g.a.c, g.a.b, g.a.n_q_heads, kCols / R), 256, lds, stream>>>(g);
  return hipGetLastError();
}

template <bool BF, int NB>
hipError_t launch_narrow(const AttnArgs &g, int R, hipStream_t stream) {
  return R == 4 ? launch_narrow<BF, NB, 4>(g, stream) : R == 2 ? launch_narrow<BF, NB, 2>(g, stream) : launch_narrow<BF, NB, 1>(g, stream);
}

}  // namespace

size_t kv4_attn_workspace_bytes(const trellis_kv4_cache &c, const trellis_kv4_batch &b, int n_q_heads) {
  // (most with whole column tiles on a full grid; fewer columns need less of each part)
  size_t most = 0;
  if (b.n_seq > 0)
    for (int C = 4; C <= kCols; C *= 2) {
      const size_t n = (size_t)narrow_grid(c, b, n_q_heads, C) * 2 * C * (c.head_dim + 8) * 4;
      most = n > most ? n : most;
    }
  return kWsReserved + most;
}

hipError_t launch_kv4_attn(const Kv4Attn &a, void *ws, hipStream_t stream) {
  AttnArgs g{};
  g.a = a;
  g.a.window = a.window < (1 << 30) ? a.window : 1 << 30;  // (longer than any sequence)
  g.a.sinks = a.sinks < (1 << 30) ? a.sinks : 1 << 30;
  g.errword = static_cast<uint32_t *>(ws);
  g.counters = reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + kWsHeaderBytes);
  g.parts = reinterpret_cast<float *>(static_cast<char *>(ws) + kWsReserved);
  g.group = a.n_q_heads / a.c.n_kv_heads;
  for (g.page_shift = 4; (1 << g.page_shift) < a.c.page_size;) ++g.page_shift;
  g.page_stride = (uint32_t)trellis_kv4_page_bytes(a.c.page_size, a.c.n_kv_heads, a.c.head_dim);
  const int R = replicas(a.c, a.b, a.n_q_heads, a.max_rows);
  const bool bf = a.dtype == TRELLIS_KV4_BF16;
  if (a.c.head_dim == 128) return bf ? launch_narrow<true, 1>(g, R, stream) : launch_narrow<false, 1>(g, R, stream);
  return bf ? launch_narrow<true, 2>(g, R, stream) : launch_narrow<false, 2>(g, R, stream);
}

}  // namespace trellis
