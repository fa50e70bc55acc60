// Attention over the 4-bit key/value cache, on the scaled matrix instructions.
//
// Mathematics.  With q' = H q (rotated once per row) a score is q . k = sum over blocks of
// ks * (q' . kc): kc the stored E2M1 codes, ks the block's scale.  The codes are matrix operands
// as they lie in memory: v_mfma_scale_f32_16x16x128_f8f6f4 takes an E2M1 operand against one of
// more bits, 128 products deep, so a key is never unpacked and its scale is one multiplication
// per score.  Likewise y' = sum_j (p_j vs_j) vc_j with the value's scale taken into the weight,
// and y = H y' at the end.
//
// Precision.  What meets the codes is split into parts, each the rounding of what the last one left: a
// query into three of E2M3 (within 2^-13.9 of the block's largest element), with one power of two per
// (row, block); a weight p_j vs_j into three of E4M3 (within 2^-14 of itself as long as it is 2^-14 of the
// tile's largest value scale, and of 2^-28 of that below: the last part's smallest step), with one power
// of two per tile of 128 keys.  Products and sums are fp32, as are the maxima, the sums of weights and
// everything that is joined.
#include "kv4_attn_device.h"

namespace trellis {

namespace {

// One wave's share of shared memory: a value tile (then, at a segment's end, its sums), and the
// tile's scales, reordered so that a lane's 32 keys are contiguous.
template <int NB, int R>
struct WaveLds {
  alignas(16) char v[NB * kCols * kRowF * 4];  // >= NB * 8 KiB
  alignas(16) uint16_t ks[NB][kTile], vs[NB][kTile];
  alignas(16) int w[R > 1 ? 4 * (kCols / R) * 3 + 1 : 1][8];  // weights' parts on their way between lanes; then zeros
};

// C columns as matrix operands, in shared memory (QueryBlock), in words of two registers.
template <int NB, int C>
struct QueryLds {
  alignas(16) v2i part[NB][3][3][4][C];
  int scale[NB][C];
  float add[NB][C];
};

// What a lane keeps of its column.
template <int NB>
struct Column {
  int scale[NB];
  float add;
  int pos;  // the column's position (-1: sees nothing)
};

// Where a tile's keys go.  The 128 keys are eight subtiles of 16, each within one page.  Lane l
// (m = l & 15, part = l >> 4) loads from subtile m >> 1 alone: of its tokens 2 j + (m & 1), j =
// 0 .. 7, the 16-byte part `part`, so one address and constant offsets serve the whole tile, and a
// wave's load covers 128 contiguous bytes of each subtile.  For the keys that is the E2M1 operand
// of product j with row m <-> key 16 (m >> 1) + 2 j + (m & 1); its result has in lane (n, g) the
// keys 32 g + 16 (i >> 1) + 2 j + (i & 1), i = 0 .. 3: over all j the keys 32 g .. 32 g + 31, and
// four consecutive keys make one word of the weights' E4M3 operand.
template <int NB>
struct Tile {
  v4i k[NB][8], v[NB][8];
  uint32_t ks[NB], vs[NB];  // scales of two tokens: first_token(l), + 1
  int page;                 // of the lane's subtile, -1: none
};

__device__ __forceinline__ int subtile_of(int lane) { return (lane & 15) >> 1; }
__device__ __forceinline__ int first_token(int lane) { return 16 * subtile_of(lane) + 8 * (lane & 1) + 2 * (lane >> 4); }

// The table's entry of the lane's subtile, not looked at yet (a look would wait for it and for
// every load before it); kNoEntry past the length.
constexpr int kNoEntry = -0x7FFFFFFF - 1;
__device__ __forceinline__ int tile_entry(const AttnArgs &g, const Seq &q, int tile) {
  const int tok = tile * kTile + 16 * subtile_of(opaque_tid() & 63);
  int e = kNoEntry;
  if (tok < q.len) e = ldg(g.a.b.table + (size_t)q.slot * g.a.b.max_pages + (tok >> g.page_shift));
  return e;
}

// `base`: the head's chunk of page 0 of the layer.  (A subtile without a page reads page 0's.)
template <int NB>
__device__ __forceinline__ void load_tile(const AttnArgs &g, int seen_from, const char *base, int tile, int entry, Tile<NB> &x) {
  const int lane = opaque_tid() & 63, T = g.a.c.page_size;
  const int tok = tile * kTile + 16 * subtile_of(lane), at = tok & (T - 1);
  x.page = (uint32_t)entry < (uint32_t)g.a.c.n_pages ? entry : -1;
  if (x.page < 0 && entry != kNoEntry && (tok + 15 >= seen_from || tok < g.a.sinks))
    kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);  // some row would see it
  const char *chunk = base + (uint64_t)(uint32_t)max(x.page, 0) * g.page_stride;
  const char *p = chunk + at * 64 + (lane & 1) * 64 + (lane >> 4) * 16;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const char *pk = p + nb * T * 64, *pv = p + (NB + nb) * T * 64;
#pragma unroll
    for (int j = 0; j < 8; ++j) x.v[nb][j] = ldg(reinterpret_cast<const v4i *>(pv + 128 * j));
#pragma unroll
    for (int j = 0; j < 8; ++j) x.k[nb][j] = ldg(reinterpret_cast<const v4i *>(pk + 128 * j));
  }
  const char *ps = chunk + 128 * NB * T + (at + 8 * (lane & 1) + 2 * (lane >> 4)) * 2;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    x.ks[nb] = ldg(reinterpret_cast<const uint32_t *>(ps + nb * T * 2));
    x.vs[nb] = ldg(reinterpret_cast<const uint32_t *>(ps + (NB + nb) * T * 2));
  }
}

// Moves a tile's values and scales to the wave's shared memory.  Keys that no row sees get
// scale zero.  The value scales are multiplied by a power of two that brings the tile's largest
// to [128, 256); vbyte is its inverse as a matrix instruction's scale byte, per block.  Returns
// whether one of them is not finite.
// A token's four 16-byte parts are permuted by bits 2 and 3 of its number, which spreads the
// transposed reads below over the banks.
template <int NB, int R>
__device__ __forceinline__ bool stage_tile(const AttnArgs &g, const Seq &q, int tile, const Tile<NB> &x, WaveLds<NB, R> &lds,
                                           int (&vbyte)[NB]) {
  const int lane = opaque_tid() & 63;
  char *const to = lds.v + subtile_of(lane) * 1024 + (lane & 1) * 64;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<v4i *>(to + (((lane >> 4) ^ (j >> 1)) * 16) + nb * 8192 + 128 * j) = x.v[nb][j];
  const int at = first_token(lane), tok = tile * kTile + at;
  const bool here = x.page >= 0;
  const uint32_t keep = ((here & (tok < q.len) & ((tok >= q.lo) | (tok < g.a.sinks))) ? 0xFFFFu : 0u) |
                        ((here & (tok + 1 < q.len) & ((tok + 1 >= q.lo) | (tok + 1 < g.a.sinks))) ? 0xFFFF0000u : 0u);
  bool odd = false;
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
    odd |= __any((w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u);
    const int e = __builtin_amdgcn_readfirstlane(max((int)(__builtin_bit_cast(uint32_t, top) >> 23), 32));
    const float f = __builtin_bit_cast(float, (uint32_t)(261 - e) << 23);
    const uint32_t fa = __builtin_bit_cast(uint32_t, a * f), fb = __builtin_bit_cast(uint32_t, b * f);
    *reinterpret_cast<uint32_t *>(&lds.vs[nb][at]) = (fa >> 16) | (fb & 0xFFFF0000u);
    vbyte[nb] = e - 7;
  }
  return odd;
}

// A lane's own keys.  With R = 16 / C columns held R times over (few columns: the matrix
// instruction is 16 wide anyway), replica r of a column takes NW = 8 / R of the lane's eight words
// of keys through the softmax: NW / 2 from r NW / 2 on in each half.
template <int R>
__device__ __forceinline__ int own_key(int lane, int w) {  // first of own word w's four keys
  constexpr int H = 4 / R;
  return 32 * (lane >> 4) + 16 * (w / H) + 4 * ((lane & 15) / (kCols / R) * H + w % H);
}
// Their scales, two words each.
template <int R>
__device__ __forceinline__ void read_scales(const uint16_t *s, uint32_t (&w)[16 / R]) {
  constexpr int H = 4 / R;
  const int lane = opaque_tid() & 63;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint16_t *p = s + own_key<R>(lane, half * H);
#pragma unroll
    for (int t = 0; t < H; ++t) {
      const v2i v = reinterpret_cast<const v2i *>(p)[t];
      w[2 * (half * H + t)] = v[0], w[2 * (half * H + t) + 1] = v[1];
    }
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

// A tile's values as the left operand of the second product: rows are elements 16 dt + (l & 15);
// the lane's depth holds the keys that the weights' E4M3 operand has there: two whole subtiles,
// read transposed.
// Tiles dt = 2 p, 2 p + 1 of block nb.
template <int NB, int R>
__device__ __forceinline__ void read_values(const WaveLds<NB, R> &lds, int nb, int p, v8i (&v)[2]) {
  const int lane = opaque_tid() & 63, r = lane & 15;
  typedef __attribute__((address_space(3))) const char lds_char;
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  lds_char *at = (lds_char *)lds.v + (4 * ((lane >> 4) & 1) + (lane >> 5)) * 1024 + r * 64 + ((p ^ (r >> 2)) * 16) + nb * 8192;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const v2i a = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_v2i *)(at + d * 8));
    const v2i b = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_v2i *)(at + d * 8 + 2048));
    v[d] = v8i{a[0], a[1], b[0], b[1], 0, 0, 0, 0};
  }
}

// Scores of a lane's own keys (own word t's key i), in powers of two.
template <int NB, int R>
__device__ __forceinline__ void scores(const v4i (&k)[NB][8], const QueryLds<NB, kCols / R> &q, const Column<NB> &col,
                                       const WaveLds<NB, R> &lds, float (&x)[8 / R][4]) {
  constexpr int NT = 8 / R, C = kCols / R, kChains = 4;
  const int lane = opaque_tid() & 63, r = (lane & 15) / C;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    uint32_t ks[16 / R];
    read_scales<R>(lds.ks[nb], ks);
    v8i part[3];
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      v2i w[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) w[k] = q.part[nb][s][k][lane >> 4][lane & (C - 1)];
      part[s] = v8i{w[0][0], w[0][1], w[1][0], w[1][1], w[2][0], w[2][1], 0, 0};
    }
    float y[NT][4];
#pragma unroll
    for (int j0 = 0; j0 < 8; j0 += kChains) {
      // several chains of three products side by side: one waits for itself
      floatx4 s[kChains];
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int c = 0; c < kChains; ++c) {
          const v4i &w = k[nb][j0 + c];
          const v8i a = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
          if (p == 0) s[c] = floatx4{0.f, 0.f, 0.f, 0.f};
          if (p == 0) s[c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, part[0], s[c], 4, 2, 0, scale_byte(0), 0, col.scale[nb]);
          if (p == 1) s[c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, part[1], s[c], 4, 2, 0, scale_byte(0), 1, col.scale[nb]);
          if (p == 2) s[c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, part[2], s[c], 4, 2, 0, scale_byte(0), 2, col.scale[nb]);
        }
      __builtin_amdgcn_sched_barrier(0);
      constexpr int H = 4 / R;
#pragma unroll
      for (int c = 0; c < kChains; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = j0 + c;
          float &z = y[(i >> 1) * H + (j >> 1) % H][2 * (j & 1) + (i & 1)];
          z = (j >> 1) / H == 0 ? s[c][i] : r == (j >> 1) / H ? s[c][i] : z;
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = scale_of(ks, t, i);
        x[t][i] = fmaf(y[t][i], s, nb ? x[t][i] : col.add);
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

// One tile into a column tile's sums.  mask: some row does not see some key of the tile; bad: bit
// 2 s of a subtile s without a page; odd: some value scale is not finite.
template <int NB, int R>
__device__ __forceinline__ void add_tile(const AttnArgs &g, int tile, bool mask, uint32_t bad, bool odd, const int (&vbyte)[NB],
                                         float (&x)[8 / R][4], const Column<NB> &col, WaveLds<NB, R> &lds, Sums<NB> &sum) {
  constexpr int NT = 8 / R, C = kCols / R, H = 4 / R;
  const int lane = opaque_tid() & 63, r = (lane & 15) / C, k = lane >> 4;
  if (mask) {
    asm volatile("");  // (a branch, not selects on every tile)
    const int k0 = tile * kTile + own_key<R>(lane, 0), rel = col.pos - k0;
    const int after = g.a.window ? rel - g.a.window : -0x40000000, sink = g.a.window ? g.a.sinks - k0 : 0;
    const uint32_t gone = bad >> (4 * k);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 16 * (t / H) + 4 * (t % H) + i;  // from k0
        x[t][i] = ((j <= rel) & ((j > after) | (j < sink)) & !((gone >> (2 * (t / H))) & 1)) ? x[t][i] : kNegInf;
      }
  }
  float top = kNegInf;
#pragma unroll
  for (int t = 0; t < NT; ++t) top = fmaxf(fmaxf(fmaxf(top, x[t][0]), fmaxf(x[t][1], x[t][2])), x[t][3]);
  if (R >= 4) top = fmaxf(top, lane_xor<4>(top));
  if (R >= 2) top = fmaxf(top, lane_xor<8>(top));
  top = max4(top);
  const float m = fmaxf(sum.m, top);
  const float mu = m == kNegInf ? 0.f : m;  // nothing seen so far
  const float alpha = __builtin_amdgcn_exp2f(sum.m - mu);
  sum.m = m;
  float add = 0.f;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[t][i] = __builtin_amdgcn_exp2f(x[t][i] - mu);
      add += x[t][i];
    }
  sum.l = fmaf(sum.l, alpha, add);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    uint32_t vs[16 / R];
    read_scales<R>(lds.vs[nb], vs);
    if (odd) {  // a hidden key's NaN must not reach the sums: no weight, no scale
      asm volatile("");
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (x[t][i] == 0.f) vs[2 * t + (i >> 1)] &= (i & 1) ? 0xFFFFu : 0xFFFF0000u;
    }
    int part[3][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = x[t][i] * scale_of(vs, t, i);
      }
      split3(w, part[0][t], part[1][t], part[2][t]);
    }
    v8i p0, p1, p2;
    if constexpr (R == 1) {
#pragma unroll
      for (int t = 0; t < 8; ++t) p0[t] = part[0][t], p1[t] = part[1][t], p2[t] = part[2][t];
    } else {
      // replica r turns from its own keys of all parts to all keys of part r
      const int h = lane & (C - 1), row = (k * C + h) * 3;
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        int *to = lds.w[row + s] + r * H;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if constexpr (R == 4) to[4 * half] = part[s][half];
          else *reinterpret_cast<v2i *>(to + 4 * half) = v2i{part[s][2 * half], part[s][2 * half + 1]};
        }
      }
      constexpr int zeros = 4 * C * 3;
      p0 = read8(lds.w[r < 3 ? row + r : zeros]);
      if constexpr (R == 2) p1 = read8(lds.w[r == 0 ? row + 2 : zeros]);
    }
    const int b0 = vbyte[nb] - (R > 1 ? 5 * r : 0);
    if (__any(alpha != 1.f))  // (rare once the first tiles are done)
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) sum.o[nb][dt] *= alpha;
    // two tiles of elements at a time, the next two's reads under way
    v8i v[2][2];
    read_values(lds, nb, 0, v[0]);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if (p < 3) read_values(lds, nb, p + 1, v[(p + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
      floatx4 &o0 = sum.o[nb][2 * p], &o1 = sum.o[nb][2 * p + 1];
      const v8i &v0 = v[p & 1][0], &v1 = v[p & 1][1];
      o0 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v0, p0, o0, 4, 0, 0, scale_byte(0), 0, b0);
      o1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v1, p0, o1, 4, 0, 0, scale_byte(0), 0, b0);
      if constexpr (R == 2) {
        o0 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v0, p1, o0, 4, 0, 0, scale_byte(0), 0, vbyte[nb] - 10);
        o1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v1, p1, o1, 4, 0, 0, scale_byte(0), 0, vbyte[nb] - 10);
      }
      if constexpr (R == 1) {
        o0 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v0, p1, o0, 4, 0, 0, scale_byte(0), 0, vbyte[nb] - 5);
        o1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v1, p1, o1, 4, 0, 0, scale_byte(0), 0, vbyte[nb] - 5);
        o0 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v0, p2, o0, 4, 0, 0, scale_byte(0), 0, vbyte[nb] - 10);
        o1 = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v1, p2, o1, 4, 0, 0, scale_byte(0), 0, vbyte[nb] - 10);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Few columns per sequence: single and drafted tokens.  Every key and value is read once and used for
// at most 16 columns, so HBM bounds long contexts in principle; what it measured (group 4, heads of
// 128): 64 ragged contexts of 300 .. 12288 tokens 95 us for 461 MB, 4.9 TB/s (a copy of the kernel that
// only loads takes the same); one token over 131071 40 us for 138 MB, 8.5 of them the join; one over
// 777 10.8 us, which is latency: the search, the queries, a tile a wave, the join.  Drafts over heads of
// 256 (12 sequences of 500 .. 9001 tokens): 39 us for 53 MB, bound by one wave a SIMD; over heads of 128 26 us.
//
// All sequences' (head, column tile, key tile) units stand in one line; each workgroup takes an
// equal stretch of it, whatever the lengths, and its four waves take the stretch's key tiles in
// turn, each with its own sums, joined in shared memory at a segment's end (a segment: one
// (sequence, head, column tile)).  A segment that several workgroups share is joined by the last
// of them to arrive, in order, so results do not depend on timing.
constexpr int kWaves = 4, kThreads = 64 * kWaves;
// The least stretch of tiles for which a segment is split: one a wave, but two where a segment has more
// than 128, as the join reads every part (8 heads, at one, two a wave: 777 tokens 11.3, 11.8 us, 3000 tokens
// 13.6, 15.4, 12000 tokens 15.8, 16.2, 30000 tokens 22.8, 20.6; eight sequences of 3000 tokens 17.3, 16.6).
constexpr int kMinChunk = kWaves, kMinChunkLong = 2 * kWaves, kLong = 128;
// What starting and ending a segment costs a workgroup, in tiles (64 ragged contexts: 106.7 us at 0,
// 100.0 at 2, 98.0 at 4, 98.3 at 6).
constexpr int kSegCost = 4;

template <int NB, int R>
struct NarrowLds {
  QueryLds<NB, kCols / R> q;
  WaveLds<NB, R> wave[kWaves];
  float ml[kWaves][2][kCols];
  long long scan[kWaves];
  long long found[2];
  int last;
};

// Exclusive prefix sum over the workgroup; *total gets the sum.
__device__ __forceinline__ long long block_prefix(long long v, long long *lds, long long *total) {
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

__device__ __forceinline__ int padded(int tiles, int least) { return (tiles + least - 1) & -least; }

__device__ __forceinline__ long long quotient(long long a, long long b) {  // of small numbers quickly
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// One segment, or the stretch of it that a workgroup has: key tiles t0 .. t1 - 1.
struct Segment {
  Seq q;
  int s, head, col0, t0, t1;
  int per;          // the segment's length in the line: its tiles after kSegCost (its tiles rounded up to whole
                    // chunks where all are)
  long long begin;  // the place of its first tile
};

// Resident waves a SIMD: two blocks need about 440 registers for a tile on its way and the sums (at 256
// some 200 are spilled).
template <int NB, int R>
constexpr int narrow_waves() { return NB == 1 ? 2 : 1; }

template <bool BF, int NB, int R>
__global__ __launch_bounds__(kThreads, (narrow_waves<NB, R>())) void kv4_attn_narrow_kernel(AttnArgs g) {
  constexpr int D = 128 * NB, C = kCols / R, kPart = C * (D + 8);
  extern __shared__ __attribute__((aligned(16))) char raw[];
  NarrowLds<NB, R> &lds = *reinterpret_cast<NarrowLds<NB, R> *>(raw);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int n_seq = g.a.b.n_seq;  // (those whose bounds are in order)
  const int G = gridDim.x, Hk = g.a.c.n_kv_heads;
  // ---- the line's length, with and without segments rounded up to whole chunks, and the
  // sequence of this workgroup's first unit
  bool whole = false;  // short contexts: whole chunks to a segment
  long long U = 0, chunk = 0, u = 0, u1 = 0, pre = 0;
  Segment c;
  c.s = -1;
  int least = kMinChunkLong;
  bool small = n_seq <= 64;
  Seq lane_seq{};  // the lane's sequence, where every wave holds all
  if (small) {  // every wave by itself, a lane a sequence
    Seq &q = lane_seq;
    int we = 0, wr = 0;
    if (lane < n_seq) q = seq_of<C>(g, lane, blockIdx.x == 0 && wave == 0 && g.tends);
    if (const uint64_t broken = __ballot(lane < n_seq && !q.ordered)) {
      n_seq = __builtin_ctzll(broken);
      if (lane >= n_seq) q = Seq{};
    }
    if (blockIdx.x == 0 && g.tends)
      clear_rest<NB, kThreads>(g, n_seq, n_seq ? __builtin_amdgcn_readlane(q.c0 + q.n, n_seq - 1) : 0);
    if (!__any(q.col_tiles && q.tiles > kLong)) least = kMinChunk;
    if (lane < n_seq) {
      const long long segs = (long long)Hk * q.col_tiles;
      const long long exact = segs * (kSegCost + q.tiles), round = segs * padded(q.tiles, least);
      small = max(exact, round) < (1 << 24);  // (so that 64 of either add up in 32 bits)
      we = small ? (int)exact : 0;
      wr = small ? (int)round : 0;
    }
    small = __all(small);
    if (small) {
      int pe = we, pr = wr;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int a = __shfl_up(pe, d, 64), b = __shfl_up(pr, d, 64);
        if (lane >= d) pe += a, pr += b;
      }
      const int exact = __builtin_amdgcn_readlane(pe, 63), round = __builtin_amdgcn_readlane(pr, 63);
      whole = round <= (long long)least * G;
      U = whole ? round : exact;
      chunk = whole ? least : ((uint32_t)exact + G - 1) / (uint32_t)G;
      u = blockIdx.x * chunk;
      u1 = min(u + chunk, U);
      if (u >= u1) return;
      const int end = whole ? pr : pe, w = whole ? wr : we;
      const uint64_t hit = __ballot(u >= end - w && u < end);
      c.s = __builtin_ctzll(hit);  // (the weights cover [0, U): one lane has it)
      pre = __builtin_amdgcn_readlane(end - w, c.s);
      c.q = seq_from(q, c.s);
    }
  }
  if (!small) {
    least = kMinChunkLong;
    long long exact, round;
    for (;;) {  // (twice where some bounds are out of order)
      exact = round = 0;
      int broken = n_seq;
      if (tid == 0) lds.last = n_seq;
      for (int s0 = 0; s0 < n_seq; s0 += kThreads) {
        long long we = 0, wr = 0, t;
        if (s0 + tid < n_seq) {
          const Seq q = seq_of<C>(g, s0 + tid, blockIdx.x == 0 && g.tends);
          if (!q.ordered) broken = min(broken, s0 + tid);
          we = (long long)Hk * q.col_tiles * (kSegCost + q.tiles);
          wr = (long long)Hk * q.col_tiles * padded(q.tiles, least);
        }
        block_prefix(we, lds.scan, &t);  // (its barriers put the store of lds.last before the minimum)
        exact += t;
        block_prefix(wr, lds.scan, &t);
        round += t;
      }
      if (broken < n_seq) atomicMin(&lds.last, broken);
      __syncthreads();
      const int ordered = __builtin_amdgcn_readfirstlane(lds.last);
      if (ordered == n_seq) break;
      n_seq = ordered;
      __syncthreads();  // lds.last is read
    }
    if (blockIdx.x == 0 && g.tends) clear_rest<NB, kThreads>(g, n_seq, n_seq ? ldg(g.a.b.cu + n_seq) : 0);
    whole = round <= (long long)least * G;
    U = whole ? round : exact;
    chunk = whole ? least : (exact + G - 1) / G;
    u = blockIdx.x * chunk;
    u1 = min(u + chunk, U);
    if (u >= u1) return;
    if (tid == 0) lds.found[0] = -1;
    __syncthreads();
    long long base = 0;
    for (int s0 = 0; s0 < n_seq && u >= base; s0 += kThreads) {
      long long w = 0, t;
      if (s0 + tid < n_seq) {
        const Seq q = seq_of<C>(g, s0 + tid, false);
        w = (long long)Hk * q.col_tiles * (whole ? padded(q.tiles, least) : kSegCost + q.tiles);
      }
      const long long p = base + block_prefix(w, lds.scan, &t);
      if (u >= p && u < p + w) lds.found[0] = s0 + tid, lds.found[1] = p;
      base += t;
    }
    __syncthreads();
    c.s = __builtin_amdgcn_readfirstlane((int)lds.found[0]);
    if (c.s < 0) return;  // (the lengths changed under the call)
    pre = lds.found[1];
    c.q = seq_from(seq_of<C>(g, c.s, false), 0);
  }
  if (c.q.col_tiles == 0) return;  // (as above)
  const int ahead = whole ? 0 : kSegCost;  // of a segment's tiles
  c.per = whole ? padded(c.q.tiles, least) : ahead + c.q.tiles;
  {
    const long long seg = quotient(u - pre, c.per);
    c.begin = pre + seg * c.per + ahead;
    c.t0 = (int)max(u - c.begin, 0LL);
    c.t1 = (int)min((long long)c.q.tiles, u1 - c.begin);
    c.head = (int)quotient(seg, c.q.col_tiles);
    c.col0 = (int)(seg - (long long)c.head * c.q.col_tiles) * C;
    if (c.t1 <= 0) return;  // (only the start of a segment that others have)
  }
  // ---- segment by segment; the next one's query, pages and first tile are on their way while this
  // one is worked on
  WaveLds<NB, R> &mine = lds.wave[wave];
  if constexpr (R > 1) {
    if (lane < 8) mine.w[4 * C * 3][lane] = 0;
  }
  Tile<NB> x;
  QueryRaw<NB> query = load_query<NB>(g, c.q, c.head, column_base(g, c.col0), tid >> 4);
  const char *base = kv4_chunk(g.a.c, g.a.layer, 0, c.head);
  {
    const int t = c.t0 + wave;
    if (t < c.t1 && c.q.len > 0) load_tile(g, c.q.lo, base, tile_at(c.q, t), tile_entry(g, c.q, tile_at(c.q, t)), x);
  }
  for (;;) {
    const Seq &q = c.q;
    const int head = c.head, col0 = c.col0;
    int t = c.t0 + wave;
    const int t1 = c.t1;
    int entry = kNoEntry, entry_n = kNoEntry;
    if (t + kWaves < t1 && q.len > 0) entry = tile_entry(g, q, tile_at(q, t + kWaves));
    // the next segment
    Segment n = c;
    n.begin = c.begin + c.per;
    bool more = n.begin < u1;
    bool first_n = false;  // this wave has a tile of it
    QueryRaw<NB> query_n = query;
    if (more) {
      n.t0 = 0;
      n.col0 += C;
      if (n.col0 >= q.col_tiles * C) {
        n.col0 = 0;
        if (++n.head == Hk) {
          n.head = 0;
          do {
            if (++n.s >= n_seq) return;  // (the lengths changed under the call)
            n.q = small ? seq_from(lane_seq, n.s) : seq_from(seq_of<C>(g, n.s, false), 0);
          } while (n.q.col_tiles == 0);
          n.per = whole ? padded(n.q.tiles, least) : ahead + n.q.tiles;
        }
      }
      n.t1 = (int)min((long long)n.q.tiles, u1 - n.begin);
      first_n = wave < n.t1 && n.q.len > 0;
      if (first_n) entry_n = tile_entry(g, n.q, tile_at(n.q, wave));
      query_n = load_query<NB>(g, n.q, n.head, column_base(g, n.col0), tid >> 4);
    }
    const char *base_n = kv4_chunk(g.a.c, g.a.layer, 0, n.head);
    {
      auto *stage = reinterpret_cast<float(*)[kCols][kRowF]>(lds.wave[0].v);  // (free between segments)
      if ((tid >> 4) < C) stage_query<BF, NB>(g, query, tid >> 4, stage);
      __syncthreads();
      if (wave < NB && (lane & 15) < C) {
        const int cc = lane & 15;
        const QueryBlock b = take_block(stage[wave][cc] + 32 * (lane >> 4));
#pragma unroll
        for (int s = 0; s < 3; ++s)
#pragma unroll
          for (int k = 0; k < 3; ++k) lds.q.part[wave][s][k][lane >> 4][cc] = v2i{(int)b.part[s][2 * k], (int)b.part[s][2 * k + 1]};
        if (lane < 16) lds.q.scale[wave][cc] = b.scale, lds.q.add[wave][cc] = b.add;
      }
      __syncthreads();
    }
    const int cols = (int)min((long long)C, (long long)q.n * g.group - col0);
    const ColumnBase from = column_base(g, col0);
    const int pos0 = q.len - q.n + from.row, pos1 = q.len - q.n + column_at(g, from, cols - 1).row;
    Column<NB> column;
    {
      const int cc = lane & (C - 1);
      column.pos = cc < cols ? q.len - q.n + column_at(g, from, cc).row : -1;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) column.scale[nb] = lds.q.scale[nb][cc];
      column.add = lds.q.add[0][cc];
      if constexpr (NB == 2) column.add += lds.q.add[1][cc];
    }
    // ---- this wave's tiles
    Sums<NB> sum;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) sum.o[nb][dt] = floatx4{0.f, 0.f, 0.f, 0.f};
    sum.m = kNegInf;
    sum.l = 0.f;
    for (;; t += kWaves) {
      const bool work = t < t1 && q.len > 0, last = t + kWaves >= t1;
      const int tile = tile_at(q, t), k0 = tile * kTile;
      uint32_t bad = 0;
      bool odd = false;
      int vbyte[NB];
      float sc[8 / R][4];
      if (work) {
        bad = (uint32_t)__ballot(x.page < 0) & 0x5555u;  // (lanes 2 s have subtile s)
        odd = stage_tile(g, q, tile, x, mine, vbyte);
        scores<NB, R>(x.k, lds.q, column, mine, sc);
      }
      __builtin_amdgcn_sched_barrier(0);  // (the next tile's loads reuse the registers of this one)
      if (!last || first_n) {
        load_tile(g, last ? n.q.lo : q.lo, last ? base_n : base, last ? tile_at(n.q, wave) : tile_at(q, t + kWaves),
                  last ? entry_n : entry, x);
        if (t + 2 * kWaves < t1) entry = tile_entry(g, q, tile_at(q, t + 2 * kWaves));
      }
      __builtin_amdgcn_sched_barrier(0);
      if (work) {
        const bool all = k0 + kTile - 1 <= pos0 && bad == 0 &&
                         (g.a.window == 0 || k0 > pos1 - g.a.window || k0 + kTile <= g.a.sinks);
        add_tile<NB, R>(g, tile, !all, bad, odd, vbyte, sc, column, mine, sum);
      }
      if (last) break;
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
    // the workgroups that share the segment
    const int w0 = (int)quotient(c.begin, chunk), w1 = (int)quotient(c.begin + q.tiles - 1, chunk);
    if (w0 == w1) {
      if ((tid >> 4) < cols)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) write_block<BF>(g, q, head, column_at(g, from, col), nb, v[nb], M, L);
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
        const int width = cols <= 1 ? 1 : cols <= 2 ? 2 : cols <= 4 ? 4 : cols <= 8 ? 8 : 16, subs = kThreads / 16 / width;
        const int sub = (tid >> 4) / width, cc = (tid >> 4) % width;
        float m = kNegInf, l2 = 0.f, acc[NB][8];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[nb][e] = 0.f;
        // the loads of several parts are in flight together (each is a trip to memory)
        constexpr int kBatch = NB == 1 ? 8 : 4;
        if (cc < cols)
          for (int w = w0 + sub; w <= w1; w += kBatch * subs) {
            u32x2 ml[kBatch];
            u32x4 p[kBatch][NB][2];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int from = min(w + k * subs, w1), at = ((from * 2 + (from == w0 ? 1 : 0)) * kPart + cc * (D + 8)) * 4;
              ml[k] = __builtin_amdgcn_raw_buffer_load_b64(rs, at + D * 4, 0, kSC1);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                p[k][nb][0] = __builtin_amdgcn_raw_buffer_load_b128(rs, at + (nb * 128 + 8 * i) * 4, 0, kSC1);
                p[k][nb][1] = __builtin_amdgcn_raw_buffer_load_b128(rs, at + (nb * 128 + 8 * i + 4) * 4, 0, kSC1);
              }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              if (w + k * subs > w1) break;
              const uint32_t mw = ml[k][0], lw = ml[k][1];
              const float pm = __builtin_bit_cast(float, mw), pl = __builtin_bit_cast(float, lw);
              const float m2 = fmaxf(m, pm), u2 = m2 == kNegInf ? 0.f : m2;
              const float fa = __builtin_amdgcn_exp2f(m - u2), fb = __builtin_amdgcn_exp2f(pm - u2);
              m = m2;
              l2 = l2 * fa + pl * fb;
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  acc[nb][e] = acc[nb][e] * fa + __builtin_bit_cast(float, (uint32_t)p[k][nb][e >> 2][e & 3]) * fb;
            }
          }
        // the shares, in order
        using W = WaveLds<NB, R>;
        static_assert(R == 1 || kThreads * (8 * NB + 2) * sizeof(float) <= offsetof(W, w) + sizeof(W::w) - sizeof(W::w[0]),
                      "the shares must leave the first wave's zeros alone");
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
        if (sub == 0 && cc < cols) {
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
          for (int nb = 0; nb < NB; ++nb) write_block<BF>(g, q, head, column_at(g, from, cc), nb, acc[nb], m, l2);
        }
      }
    }
    if (!more) break;
    c = n;
    query = query_n;
    base = base_n;
    __syncthreads();  // shared memory is free again
  }
}

// How often the narrow kernel holds a column: as many columns as the sequences' rows are known or
// expected to have, up to 4, 8 or 16 a tile (group 4, by this rule and with 16 throughout: one
// token over 131071 39.7, 43.4 us, over 777 13.6, 15.6; 64 ragged contexts 99, 102; two tokens each
// over 777 14.3, 15.4, 64 ragged contexts 103.9, 104.2).
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
  const long long most = (long long)micro_cus() * (c.head_dim == 128 ? narrow_waves<1, 1>() : narrow_waves<2, 1>());
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
  kernel<<<narrow_grid(g.a.c, g.a.b, g.a.n_q_heads, kCols / R), kThreads, lds, stream>>>(g);
  return hipGetLastError();
}

template <bool BF, int NB>
hipError_t launch_narrow(const AttnArgs &g, int R, hipStream_t stream) {
  return R == 4 ? launch_narrow<BF, NB, 4>(g, stream) : R == 2 ? launch_narrow<BF, NB, 2>(g, stream) : launch_narrow<BF, NB, 1>(g, stream);
}

}  // namespace

size_t kv4_attn_workspace_bytes(const trellis_kv4_cache &c, const trellis_kv4_batch &b, int n_q_heads) {
  // (most with whole column tiles on a full grid; fewer columns need less of each part)
  size_t most = kv4_attn_wide_parts(c, b, n_q_heads);
  if (b.n_seq > 0)
    for (int C = 4; C <= kCols; C *= 2) {
      const size_t n = (size_t)narrow_grid(c, b, n_q_heads, C) * 2 * C * (c.head_dim + 8) * 4;
      most = n > most ? n : most;
    }
  return kWsReserved + most;
}

// A sequence of at most this many columns (rows times query heads per key/value head) is the
// narrow kernel's, whose tiles are 16 columns wide and shared by any number of workgroups; the
// wide kernel's are 64.  Narrow against wide, in us: 16 sequences of 3000 .. 6000 tokens, heads of 128,
// 32 columns 40, 48, 48 columns 51, 58, 64 columns 60, 62, 96 columns 81, 85, 128 columns 102, 88; 64 such
// sequences, 48 columns 182, 144; 8 of heads of 256, 32 columns 39, 49, 48 columns 49, 52, 64 columns 59, 50.
// A single sequence has few wide segments, which have to be split and joined: 30000 tokens, 64 columns
// 38, 53, 128 columns 52, 54, 192 columns 67, 71, 256 columns 80, 72.
int few_columns(int n_seq) { return n_seq == 1 ? 128 : 48; }

hipError_t launch_kv4_attn(const Kv4Attn &a, void *ws, hipStream_t stream) {
  AttnArgs g{};
  g.a = a;
  g.a.window = a.window < (1 << 30) ? a.window : 1 << 30;  // (longer than any sequence)
  g.a.sinks = a.sinks < (1 << 30) ? a.sinks : 1 << 30;
  g.errword = static_cast<uint32_t *>(ws);
  g.counters = reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + kWsHeaderBytes);
  g.parts = reinterpret_cast<float *>(static_cast<char *>(ws) + kWsReserved);
  g.group = a.n_q_heads / a.c.n_kv_heads;
  g.per_group = 65536 / g.group + 1;
  for (g.page_shift = 4; (1 << g.page_shift) < a.c.page_size;) ++g.page_shift;
  g.page_stride = (uint32_t)trellis_kv4_page_bytes(a.c.page_size, a.c.n_kv_heads, a.c.head_dim);
  // Which kernels: one where every sequence is known to be its kind (that kernel then takes whatever
  // there is, so a wrong bound costs time and nothing else), otherwise both, each with its sequences.
  const long long bound = (long long)(a.b.n_seq == 1 ? a.b.rows : a.max_rows > 0 ? a.max_rows : a.b.rows) * g.group;
  const int few = few_columns(a.b.n_seq);
  const bool both = a.b.n_seq > 1 && bound > few;
  g.tends = 1;
  if (both) {
    g.few = few;
    const hipError_t e = launch_kv4_attn_wide(g, stream);
    if (e != hipSuccess) return e;
    g.tends = 0;
  } else if (bound > few) {
    g.few = -1;
    return launch_kv4_attn_wide(g, stream);
  } else {
    g.few = 0x7FFFFFFF;
  }
  const int R = replicas(a.c, a.b, a.n_q_heads, both ? 0 : a.max_rows);
  const bool bf = a.dtype == TRELLIS_KV4_BF16;
  if (a.c.head_dim == 128) return bf ? launch_narrow<true, 1>(g, R, stream) : launch_narrow<false, 1>(g, R, stream);
  return bf ? launch_narrow<true, 2>(g, R, stream) : launch_narrow<false, 2>(g, R, stream);
}

}  // namespace trellis
