// Attention over the 4-bit key/value cache, many columns per sequence: prompts and chunks of them.
// (Mathematics and formats: kv4_attn.hip.)
//
// A workgroup takes 64 columns (rows times the query heads of one key/value head) of one sequence,
// 16 a wave, and walks its key tiles of 128.  A tile is copied to shared memory once for all four
// waves, into two buffers in turn, with one barrier a tile.
//
// Scores are as in the narrow kernel: codes against three parts of the query.  The second product is
// different: per column a tile's three-way split of the weights costs as many
// vector instructions as turning the values to fp16 does, and its products twice the time.  So a
// value tile's codes are read transposed and turned to fp16 in registers (exactly), and the weights
// p vs are rounded once to fp16 (within 2^-11), with one power of two per wave that follows the
// tiles' largest value scale.
//
// Issue bounds it: 586 vector instructions a tile and wave with starts and ends, 128 of them the values'
// conversion, keep a SIMD busy 75% of the time, and the matrix instructions (900 cycles a tile and wave at
// heads of 128) run beside them but take slots too.  Three waves a SIMD overlap them; more columns a wave
// would share the conversion, but leave two waves (32 a wave: 374 us where 64 columns a workgroup took 245).
// 4096 tokens, 32 query heads, 8 key/value heads of 128: 182 us, 137 GFLOP, 755 TFLOP/s (the library's fp16
// product of 8192^3 reaches 1330); copies that leave work out take 160 us without the conversion, 170 with
// one of the query's three parts, 144 with a quarter of the second product.  16 query heads on 4 of 256:
// 183 us.  Chunks of 300 .. 1023 tokens behind up to 11000, window 2048: 92 us, 39 GFLOP.
#include "kv4_attn_device.h"

namespace trellis {

namespace {

constexpr int kWideCols = 64, kWideThreads = 256;  // 16 columns a wave

constexpr uint32_t kOdd = 1, kBad = 2;  // a value scale is not finite; the subtile has no page

template <int NB>
struct WideTiles {
  alignas(16) char k[2][NB][8192], v[2][NB][8192];
  alignas(16) float ks[2][NB][kTile], vs[2][NB][kTile];
  alignas(16) uint32_t about[2][NB][8];  // subtiles: the largest finite value scale's exponent << 8 | kOdd | kBad
};
template <int NB>
union WideLds {
  WideTiles<NB> t;
  float o[4][NB][kCols][kRowF];       // before the tiles queries, after them sums: one column tile a wave
  int last;
};

// A tile's way to shared memory: each wave copies two of its eight subtiles of 16 tokens, 1024
// contiguous bytes of keys and of values for each block, with copies that pass by the registers.
// The scales go through registers, where those of keys that no row sees become zero: half a
// wave has a subtile's, two tokens a lane.
struct Share {
  uint32_t s;  // lanes 0..7 of a subtile key scales, 8..15 value scales (16..31: block 1)
  int page;
};

constexpr int kNoPage = -0x7FFFFFFF - 1;  // past the length
__device__ __forceinline__ int share_entry(const AttnArgs &g, const Seq &q, int tile) {
  const int tok = tile * kTile + 16 * (threadIdx.x >> 5);
  int e = kNoPage;
  if (tok < q.len) e = ldg(g.a.b.table + (size_t)q.slot * g.a.b.max_pages + (tok >> g.page_shift));
  return e;
}

// The 16-byte parts of a tile in shared memory are permuted so that the products' reads spread over
// the banks: key parts by their subtile (a product reads two tokens of each subtile), value parts by
// bits 2 and 3 of their token.
__device__ __forceinline__ int key_swizzle(int subtile) { return (subtile & 3) | ((subtile & 4) << 1); }

// (A subtile without a page copies page 0's, whose scales become zero.)  The copies are not waited
// for by anything but an explicit wait.
template <int NB>
__device__ __forceinline__ void load_share(const AttnArgs &g, int lo, const char *base, int tile, int entry, WideTiles<NB> &lds, int buf,
                                           Share &x) {
  const int T = g.a.c.page_size, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  {
    const int tok = tile * kTile + 16 * (threadIdx.x >> 5), i = threadIdx.x & 31;
    x.page = (uint32_t)entry < (uint32_t)g.a.c.n_pages ? entry : -1;
    if (x.page < 0 && entry != kNoPage && (tok + 15 >= lo || tok < g.a.sinks)) kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);
    const char *chunk = base + (uint64_t)(uint32_t)max(x.page, 0) * g.page_stride;
    x.s = 0;
    const int nb = i >> 4, kind = (i >> 3) & 1, at = tok & (T - 1);
    if (nb < NB) x.s = ldg(reinterpret_cast<const uint32_t *>(chunk + 128 * NB * T + ((kind * NB + nb) * T + at + 2 * (i & 7)) * 2));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int sub = 2 * wave + h, at = (tile * kTile + 16 * sub) & (T - 1);
    const int page = max(__builtin_amdgcn_readlane(x.page, 32 * h), 0);
    const char *p = base + (uint64_t)(uint32_t)page * g.page_stride + at * 64;
    typedef __attribute__((address_space(1))) const void gbl_void;
    typedef __attribute__((address_space(3))) void lds_void;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const char *k = p + nb * T * 64 + (lane ^ key_swizzle(sub)) * 16, *v = p + (NB + nb) * T * 64 + (lane ^ ((lane >> 4) & 3)) * 16;
      __builtin_amdgcn_global_load_lds((gbl_void *)k, (lds_void *)(lds.k[buf][nb] + sub * 1024), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((gbl_void *)v, (lds_void *)(lds.v[buf][nb] + sub * 1024), 16, 0, 0);
    }
  }
}

template <int NB>
__device__ __forceinline__ void put_share(const AttnArgs &g, const Seq &q, int tile, const Share &x, WideTiles<NB> &lds, int buf) {
  const int s = threadIdx.x >> 5, i = threadIdx.x & 31;
  const int nb = i >> 4, kind = (i >> 3) & 1, at = 16 * s + 2 * (i & 7), tok = tile * kTile + at;
  if (nb < NB) {
    const bool here = x.page >= 0;
    const uint32_t keep = ((here & (tok < q.len) & ((tok >= q.lo) | (tok < g.a.sinks))) ? 0xFFFFu : 0u) |
                          ((here & (tok + 1 < q.len) & ((tok + 1 >= q.lo) | (tok + 1 < g.a.sinks))) ? 0xFFFF0000u : 0u);
    const uint32_t w = x.s & keep;
    float *to = kind ? lds.vs[buf][nb] : lds.ks[buf][nb];
    *reinterpret_cast<floatx2 *>(to + at) = floatx2{__builtin_bit_cast(float, w << 16), __builtin_bit_cast(float, w & 0xFFFF0000u)};
    // the eight lanes' largest, as bf16's bits without sign
    const uint32_t a = w & 0x7FFFu, b = (w >> 16) & 0x7FFFu;
    const bool fa = a < 0x7F80u, fb = b < 0x7F80u;
    uint32_t top = (max(fa ? a : 0u, fb ? b : 0u) << 1) & ~0xFFu;  // its exponent << 8
    top |= ((fa & fb) ? 0 : kOdd) | (here ? 0 : kBad);
    const auto merge = [](uint32_t x, uint32_t y) { return max(x & ~0xFFu, y & ~0xFFu) | ((x | y) & 0xFFu); };
    top = merge(top, __builtin_amdgcn_update_dpp(0, top, 0xB1, 0xF, 0xF, true));
    top = merge(top, __builtin_amdgcn_update_dpp(0, top, 0x4E, 0xF, 0xF, true));
    top = merge(top, __builtin_amdgcn_update_dpp(0, top, 0x141, 0xF, 0xF, true));
    if (kind && (i & 7) == 0) lds.about[buf][nb][s] = top;
  }
}

// A lane's 32 keys' scales (32 g .. 32 g + 31).
__device__ __forceinline__ void read_scales32(const float *s, float (&w)[32]) {
  const floatx4 *p = reinterpret_cast<const floatx4 *>(s + ((threadIdx.x & 63) >> 4) * 32);
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const floatx4 v = p[t];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[4 * t + e] = v[e];
  }
}
// Key (j, i) of the products' results is key 16 (i >> 1) + 2 j + (i & 1) of the lane's.
__device__ __forceinline__ constexpr int key32(int j, int i) { return 16 * (i >> 1) + 2 * j + (i & 1); }

// A wave's 16 columns as matrix operands (QueryBlock).
template <int NB>
struct Query {
  v8i part[NB][3];  // (six registers each)
  int scale[NB];
  float add;
};

template <int NB>
__device__ __forceinline__ void take_query(const float (&from)[NB][kCols][kRowF], Query<NB> &q) {
  const int lane = threadIdx.x & 63;
  q.add = 0.f;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const QueryBlock b = take_block(from[nb][lane & 15] + 32 * (lane >> 4));
#pragma unroll
    for (int s = 0; s < 3; ++s)
      q.part[nb][s] = v8i{(int)b.part[s][0], (int)b.part[s][1], (int)b.part[s][2], (int)b.part[s][3], (int)b.part[s][4], (int)b.part[s][5], 0, 0};
    q.scale[nb] = b.scale;
    q.add += b.add;
  }
}

// A lane's codes of a value tile's block, read transposed: tile dt = 2 p + d, 1024-byte half h.  One block
// with its wait: for the builtin the compiler also waits for every copy to shared memory that is under
// way, the next tile's among them.
__device__ __forceinline__ void read_codes(const char *vp, int swizzle, v2i (&c)[4][2][2]) {
  typedef __attribute__((address_space(3))) const char lds_char;
  const uint32_t at = (uint32_t)(uintptr_t)(lds_char *)vp;
  const uint32_t a0 = at + swizzle * 16, a1 = at + (1 ^ swizzle) * 16, a2 = at + (2 ^ swizzle) * 16, a3 = at + (3 ^ swizzle) * 16;
  asm volatile(
      "ds_read_b64_tr_b4 %0, %16\n\tds_read_b64_tr_b4 %1, %16 offset:1024\n\t"
      "ds_read_b64_tr_b4 %2, %16 offset:8\n\tds_read_b64_tr_b4 %3, %16 offset:1032\n\t"
      "ds_read_b64_tr_b4 %4, %17\n\tds_read_b64_tr_b4 %5, %17 offset:1024\n\t"
      "ds_read_b64_tr_b4 %6, %17 offset:8\n\tds_read_b64_tr_b4 %7, %17 offset:1032\n\t"
      "ds_read_b64_tr_b4 %8, %18\n\tds_read_b64_tr_b4 %9, %18 offset:1024\n\t"
      "ds_read_b64_tr_b4 %10, %18 offset:8\n\tds_read_b64_tr_b4 %11, %18 offset:1032\n\t"
      "ds_read_b64_tr_b4 %12, %19\n\tds_read_b64_tr_b4 %13, %19 offset:1024\n\t"
      "ds_read_b64_tr_b4 %14, %19 offset:8\n\tds_read_b64_tr_b4 %15, %19 offset:1032\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(c[0][0][0]), "=&v"(c[0][0][1]), "=&v"(c[0][1][0]), "=&v"(c[0][1][1]), "=&v"(c[1][0][0]), "=&v"(c[1][0][1]),
        "=&v"(c[1][1][0]), "=&v"(c[1][1][1]), "=&v"(c[2][0][0]), "=&v"(c[2][0][1]), "=&v"(c[2][1][0]), "=&v"(c[2][1][1]),
        "=&v"(c[3][0][0]), "=&v"(c[3][0][1]), "=&v"(c[3][1][0]), "=&v"(c[3][1][1])
      : "v"(a0), "v"(a1), "v"(a2), "v"(a3)
      : "memory");
}

// By how many powers of two a wave's sums of a block can grow and stay below 2^126, so that later tiles
// (2^42 at most, all together) still add up to a finite number.  Sums that are not finite stay so.
__device__ __forceinline__ int sums_room(const floatx4 (&o)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int dt = 0; dt < 8; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = o[dt][i];
      const uint32_t u = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
      top = max(top, u < 0x7F800000u ? u : 0u);
    }
  top = max4u(kv4_max16(top));
  return max(252 - (int)(__builtin_amdgcn_readfirstlane(top) >> 23), 0);
}

// One tile into a wave's sums.  mask: some row does not see some key; bad: subtiles without a page;
// odd: some value scale is not finite.
template <int NB>
__device__ __forceinline__ void wide_tile(const AttnArgs &g, const WideTiles<NB> &lds, int buf, int k0, bool mask, uint32_t bad, bool odd,
                                          const Query<NB> &query, int pos, const float (&f)[NB], const int (&e_run)[NB], float &m,
                                          float &l, floatx4 (&o)[NB][8]) {
  const int lane = opaque_tid() & 63;
  const float log2f = (float)max(134 - e_run[0], -60);  // (2^-60: weights stay far from the smallest number)
  half8 w[NB][4];
  // ---- scores, from the running maximum (or from 0) as the weights' powers of two
  const float mu = m == kNegInf ? 0.f : m, c0 = log2f - mu + query.add;
  float y[8][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    // Products j = 2 p, 2 p + 1 together.  The order is kept as written: the next two's keys are
    // on their way during the products, and two chains of three products alternate; left to
    // itself the compiler waits for every load and every product.
    const int row = lane & 15, sub = row >> 1;
    const char *kp = lds.k[buf][nb] + sub * 1024;
    const float *sp = lds.ks[buf][nb] + (lane >> 4) * 32;
    v4i kv[2][2];
    floatx4 s4[2][2], z[2][2];
    const auto load = [&](int p) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = (8 * h + 4 * (row & 1) + (lane >> 4)) ^ key_swizzle(sub);
        kv[p & 1][h] = *reinterpret_cast<const v4i *>(kp + p * 256 + c * 16);
      }
    };
    load(0);
#pragma unroll
    for (int p = 0; p < 5; ++p) {
      const int at = p & 1;
      if (p < 4) {
        if (p < 3) load(p + 1);
        // keys 4 p .. + 3 and 16 + 4 p .. + 3 of the lane's
        s4[at][0] = *reinterpret_cast<const floatx4 *>(sp + 4 * p);
        s4[at][1] = *reinterpret_cast<const floatx4 *>(sp + 16 + 4 * p);
        __builtin_amdgcn_sched_barrier(0);
        const v8i a0 = {kv[at][0][0], kv[at][0][1], kv[at][0][2], kv[at][0][3], 0, 0, 0, 0};
        const v8i a1 = {kv[at][1][0], kv[at][1][1], kv[at][1][2], kv[at][1][3], 0, 0, 0, 0};
        const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
        const int scale = query.scale[nb];
        z[at][0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a0, query.part[nb][0], zero, 4, 2, 0, scale_byte(0), 0, scale);
        z[at][1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a1, query.part[nb][0], zero, 4, 2, 0, scale_byte(0), 0, scale);
        z[at][0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a0, query.part[nb][1], z[at][0], 4, 2, 0, scale_byte(0), 1, scale);
        z[at][1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a1, query.part[nb][1], z[at][1], 4, 2, 0, scale_byte(0), 1, scale);
        z[at][0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a0, query.part[nb][2], z[at][0], 4, 2, 0, scale_byte(0), 2, scale);
        z[at][1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a1, query.part[nb][2], z[at][1], 4, 2, 0, scale_byte(0), 2, scale);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (p > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float &to = y[2 * (p - 1) + h][i];
            to = fmaf(z[at ^ 1][h][i], s4[at ^ 1][i >> 1][2 * h + (i & 1)], nb ? to : c0);
          }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // ---- softmax
  if (mask) {
    asm volatile("");  // (a branch, not 32 selects on every tile)
    const int kk = k0 + 32 * (lane >> 4), rel = pos - kk;
    const int after = g.a.window ? rel - g.a.window : -0x40000000, sink = g.a.window ? g.a.sinks - kk : 0;
    const uint32_t gone = bad >> (2 * (lane >> 4));
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 16 * (i >> 1) + 2 * j + (i & 1);
        y[j][i] = ((k <= rel) & ((k > after) | (k < sink)) & !((gone >> (i >> 1)) & 1)) ? y[j][i] : kNegInf;
      }
  }
  // The running maximum stays until a lane's weights outgrow 2^7 together: most tiles then need
  // neither a maximum nor a rescaling.  The power of two f[0] is taken into the exponent.
  float add = 0.f, alpha = 1.f;
  float x[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[j][i] = __builtin_amdgcn_exp2f(y[j][i]);
      add += x[j][i];
    }
  const float one = __builtin_amdgcn_exp2f(log2f);  // a weight of 1
  if (__any(!(add <= 128.f * one) | (m == kNegInf))) {
    float top = kNegInf;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(fmaxf(fmaxf(top, y[j][0]), fmaxf(y[j][1], y[j][2])), y[j][3]);
    top = max4(top);
    // By how much the maximum grows (where there was none, from 0).  A column that does not need it
    // stays as it is, so that no column's result depends on which others are beside it.
    const bool first = m == kNegInf, need = max4u(!(add <= 128.f * one) | first) != 0;
    const float by = first ? top - log2f : need ? fmaxf(top - log2f, 0.f) : 0.f, up = by == kNegInf ? 0.f : by;
    alpha = first ? 0.f : __builtin_amdgcn_exp2f(-up);
    m = first ? by : m + up;
    add = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[j][i] = __builtin_amdgcn_exp2f(y[j][i] - up);
        add += x[j][i];
      }
  }
  l = fmaf(l, alpha, add * __builtin_amdgcn_exp2f(-log2f));
  // ---- weights
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float vs[32];
    read_scales32(lds.vs[buf][nb], vs);
    if (nb == 0 && e_run[0] > 194) {  // what the exponent's bound left
      asm volatile("");
      const float rest = f[0] * __builtin_amdgcn_exp2f(-log2f);
#pragma unroll
      for (int k = 0; k < 32; ++k) vs[k] *= rest;
    }
    // Block 1 turns from block 0's power of two to its own: in one factor where that neither leaves a
    // float's range nor lets x vs leave it, otherwise its own first.
    float turn = 1.f;
    if (nb) {
      const int own = 134 - e_run[nb], by = own - max(134 - e_run[0], -60);
      turn = __builtin_bit_cast(float, (uint32_t)(127 + min(max(by, -60), 60)) << 23);
      if (by < -60 || by > 60) {
        asm volatile("");
        turn = __builtin_amdgcn_exp2f(-log2f);
#pragma unroll
        for (int k = 0; k < 32; ++k) vs[k] *= f[nb];
      }
    }
    if (odd) {  // a hidden key's NaN must not reach the sums: no weight, no scale
      asm volatile("");
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) vs[key32(j, i)] = x[j][i] == 0.f ? 0.f : vs[key32(j, i)];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float u = x[j][i] * vs[key32(j, i)];
        if (nb) u *= turn;
        // step 2 (i >> 1) + (j >> 2), element 2 (j & 3) + (i & 1)
        w[nb][2 * (i >> 1) + (j >> 2)][2 * (j & 3) + (i & 1)] = (_Float16)u;
      }
    if (__any(alpha != 1.f))
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) o[nb][dt] *= alpha;
  }
  __builtin_amdgcn_sched_barrier(0);  // (keeps the phases' registers apart)
  // ---- values
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int row = lane & 15, sub = 2 * (lane >> 4);
    const char *vp = lds.v[buf][nb] + sub * 1024 + row * 64;
    // Elements' tiles dt = 2 p, 2 p + 1 together, and the next word's codes turned to fp16 during
    // a word's products.
    v2i codes[4][2][2];
    read_codes(vp, row >> 2, codes);
    half8 a[2][2];
    const auto unpack = [&](int step) {  // word step & 3 of pair step >> 2
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const uint32_t c = codes[step >> 2][d][(step >> 1) & 1][step & 1];
        const half2_t a0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.f, 0), a1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.f, 1);
        const half2_t a2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.f, 2), a3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.f, 3);
        a[step & 1][d] = half8{a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
      }
    };
    unpack(0);
#pragma unroll
    for (int step = 0; step < 16; ++step) {
      const int p = step >> 2;
      if (step < 15) unpack(step + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < 2; ++d)
        o[nb][2 * p + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[step & 1][d], w[nb][step & 3], o[nb][2 * p + d], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

template <int NB>
constexpr int wide_waves() { return NB == 1 ? 3 : 2; }  // a SIMD

template <bool BF, int NB>
__global__ __launch_bounds__(kWideThreads, (wide_waves<NB>())) void kv4_attn_wide_kernel(AttnArgs g) {
  constexpr int D = 128 * NB;
  extern __shared__ __attribute__((aligned(16))) char raw[];
  WideLds<NB> &lds = *reinterpret_cast<WideLds<NB> *>(raw);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int Hk = g.a.c.n_kv_heads;
  int n_seq = g.a.b.n_seq;  // (those whose bounds are in order)
  if (n_seq > 64) {
    int broken = n_seq;
#pragma unroll 4
    for (int r = lane; r < n_seq; r += 64)
      if (!bounds_ok(g, r, ldg(g.a.b.cu + r), ldg(g.a.b.cu + r + 1))) broken = min(broken, r);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) broken = min(broken, __shfl_xor(broken, d, 64));
    n_seq = __builtin_amdgcn_readfirstlane(broken);
  }
  // ---- which columns: the last sequence's last ones first, as they see the most keys.  The head
  // varies fastest: with eight of them each XCD's cache has one head's keys.
  const int split = blockIdx.x % g.splits, head = blockIdx.x / g.splits % Hk;
  int item = blockIdx.x / g.splits / Hk, s = -1;
  Seq q{};
  for (int s1 = n_seq; s1 > 0 && s < 0; s1 -= 64) {  // 64 sequences at a time, a lane a sequence
    const int mine = s1 - 1 - lane;
    Seq x{};
    int tiles = 0;
    if (mine >= 0) {
      x = seq_of<kWideCols>(g, mine, blockIdx.x == 0 && wave == 0 && g.tends);
      tiles = x.col_tiles;
    }
    if (const uint64_t broken = __ballot(mine >= 0 && !x.ordered)) {  // (64 sequences or fewer)
      n_seq = s1 - 64 + __builtin_clzll(broken);
      if (mine >= n_seq) tiles = x.col_tiles = 0;
    }
    int p = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int a = __shfl_up(p, d, 64);
      if (lane >= d) p += a;
    }
    const uint64_t hit = __ballot(item < p);
    if (hit && s < 0) {
      const int l = __builtin_ctzll(hit);
      s = s1 - 1 - l;
      q = seq_from(x, l);
      item -= __builtin_amdgcn_readlane(p, l) - q.col_tiles;
    }
    if (s < 0) item -= __builtin_amdgcn_readlane(p, 63);
    if (blockIdx.x == 0 && g.tends && s >= 0 && s1 > 64)  // (the rest only to be checked)
      for (int r = s1 - 64 - 1 - lane; wave == 0 && r >= 0; r -= 64) seq_of<kWideCols>(g, r, true);
  }
  if (blockIdx.x == 0 && g.tends) clear_rest<NB, kWideThreads>(g, n_seq, n_seq ? ldg(g.a.b.cu + n_seq) : 0);
  if (s < 0) return;
  const int col0 = (q.col_tiles - 1 - item) * kWideCols;
  const int cols = (int)min((long long)kWideCols, (long long)q.n * g.group - col0);
  const ColumnBase from = column_base(g, col0);
  const int p0 = q.len - q.n + from.row, p1 = q.len - q.n + column_at(g, from, cols - 1).row;  // positions
  // the key tiles of these rows
  q.lo = g.a.window ? max(p0 - g.a.window + 1, 0) : 0;
  q.first = q.lo / kTile;
  q.n_sink = min((min(g.a.sinks, q.len) + kTile - 1) / kTile, q.first);
  q.tiles = max(q.n_sink + (min(max(p1 + 1, 0), q.len) + kTile - 1) / kTile - q.first, 0);
  const int t0 = (int)((long long)q.tiles * split / g.splits), t1 = (int)((long long)q.tiles * (split + 1) / g.splits);
  const char *base = kv4_chunk(g.a.c, g.a.layer, 0, head);
  // ---- queries
  Share x;
  int entry = 0;
  if (t0 < t1) entry = share_entry(g, q, tile_at(q, t0));
  Query<NB> query;
  QueryRaw<NB> r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = load_query<NB>(g, q, head, from, wave * kCols + 4 * k + (lane >> 4));
#pragma unroll
  for (int k = 0; k < 4; ++k) stage_query<BF, NB>(g, r[k], 4 * k + (lane >> 4), lds.o[wave]);
  __builtin_amdgcn_wave_barrier();
  take_query<NB>(lds.o[wave], query);
  const int mine = wave * kCols + (lane & 15);
  const int pos = mine < cols ? q.len - q.n + column_at(g, from, mine).row : -1;  // -1: sees nothing
  __syncthreads();
  floatx4 o[NB][8];
  float m, l;
  int e_run[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int dt = 0; dt < 8; ++dt) o[nb][dt] = floatx4{0.f, 0.f, 0.f, 0.f};
  m = pos < 0 ? 0.f : kNegInf;  // (a column past the last never sees a score)
  l = 0.f;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) e_run[nb] = 127;
  if (t0 < t1) load_share(g, q.lo, base, tile_at(q, t0), entry, lds.t, 0, x);
  if (t0 + 1 < t1) entry = share_entry(g, q, tile_at(q, t0 + 1));
  const int wp0 = q.len - q.n + column_at(g, from, min(wave * kCols, cols - 1)).row;
  const int wp1 = q.len - q.n + column_at(g, from, min((wave + 1) * kCols, cols)).row;  // (one more at most)
  const bool idle = wave * kCols >= cols;  // no column of this wave's
  for (int t = t0; t < t1; ++t) {
    const int buf = (t - t0) & 1, tile = tile_at(q, t), k0 = tile * kTile;
    put_share(g, q, tile, x, lds.t, buf);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's copies have arrived
    __syncthreads();                     // this tile is complete, and the one before it is read
    if (t + 1 < t1) load_share(g, q.lo, base, tile_at(q, t + 1), entry, lds.t, buf ^ 1, x);
    if (t + 2 < t1) entry = share_entry(g, q, tile_at(q, t + 2));
    if (!idle && k0 <= wp1) {
      // ---- the value scales' power of two: the tile's largest finite one comes below 2^8; it stays
      // unless the tiles' scales outgrow it or fall far below, and falls no further than the sums can
      // grow (a tile of zeros, which has no size, leaves it alone)
      float f[NB];
      uint32_t flags = 0;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        uint32_t top = 0, any = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 v = *reinterpret_cast<const u32x4 *>(lds.t.about[buf][nb] + 4 * h);
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, v[k]), any |= v[k];
        }
        flags |= any;
        const int seen = (int)(__builtin_amdgcn_readfirstlane(top) >> 8), e = max(seen, 32);
        if (seen != 0 && (e > e_run[nb] || e < e_run[nb] - 8)) {
          asm volatile("");
          int by = e_run[nb] - min(e + 2, 254);
          if (by > 0) by = min(by, sums_room(o[nb]));
          e_run[nb] -= by;
#pragma unroll
          for (int dt = 0; dt < 8; ++dt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nb][dt][i] = __builtin_ldexpf(o[nb][dt][i], by);
        }
        f[nb] = __builtin_bit_cast(float, (uint32_t)(261 - e_run[nb]) << 23);
      }
      flags = __builtin_amdgcn_readfirstlane(flags);
      const bool odd = flags & kOdd;
      uint32_t bad = 0;
      if (flags & kBad) bad = (uint32_t)__ballot(lane < 8 && (lds.t.about[buf][0][lane & 7] & kBad));
      const bool mask = !(k0 + kTile - 1 <= wp0 && bad == 0 &&
                          (g.a.window == 0 || k0 > wp1 - g.a.window || k0 + kTile <= g.a.sinks));
      wide_tile<NB>(g, lds.t, buf, k0, mask, bad, odd, query, pos, f, e_run, m, l, o);
    }
  }
  // ---- results: back to the values' units, through shared memory, 16 lanes a column
  l = sum4(l);
  __syncthreads();
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const float f = __builtin_bit_cast(float, (uint32_t)max(e_run[nb] - 7, 1) << 23);
#pragma unroll
    for (int dt = 0; dt < 8; ++dt)
      *reinterpret_cast<floatx4 *>(&lds.o[wave][nb][lane & 15][16 * dt + 4 * (lane >> 4)]) = o[nb][dt] * f;
  }
  __builtin_amdgcn_wave_barrier();
  const int i = lane & 15;
  for (int p = 0; p < 4; ++p) {
    const int c = 4 * p + (lane >> 4), at = wave * kCols + c;
    const float mm = __shfl(m, c, 64), ll = __shfl(l, c, 64);
    if (at >= cols) continue;  // (16 lanes together)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const floatx4 a = *reinterpret_cast<const floatx4 *>(&lds.o[wave][nb][c][8 * i]);
      const floatx4 b = *reinterpret_cast<const floatx4 *>(&lds.o[wave][nb][c][8 * i + 4]);
      float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      if (g.splits == 1) {
        write_block<BF>(g, q, head, column_at(g, from, at), nb, v, mm, ll);
      } else {
        const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(g.parts + (size_t)(blockIdx.x / g.splits) * g.splits * kWideCols * (D + 8),
                                                      (long long)g.splits * kWideCols * (D + 8) * 4);
        const int to = ((split * kWideCols + at) * (D + 8)) * 4;
        const u32x4 x0 = {__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]), __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3])};
        const u32x4 x1 = {__builtin_bit_cast(uint32_t, v[4]), __builtin_bit_cast(uint32_t, v[5]), __builtin_bit_cast(uint32_t, v[6]), __builtin_bit_cast(uint32_t, v[7])};
        __builtin_amdgcn_raw_buffer_store_b128(x0, rs, to + (nb * 128 + 8 * i) * 4, 0, kSC1);
        __builtin_amdgcn_raw_buffer_store_b128(x1, rs, to + (nb * 128 + 8 * i + 4) * 4, 0, kSC1);
        if (nb == 0 && i == 0)
          __builtin_amdgcn_raw_buffer_store_b64(u32x2{__builtin_bit_cast(uint32_t, mm), __builtin_bit_cast(uint32_t, ll)}, rs, to + D * 4, 0, kSC1);
      }
    }
  }
  if (g.splits == 1) return;
  // ---- the join, by the last of the segment's workgroups
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): every thread's stores have completed
  __syncthreads();
  const int seg = blockIdx.x / g.splits;
  if (tid == 0) {
    const uint32_t old = __hip_atomic_fetch_add(g.counters + seg, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    lds.last = old == (uint32_t)(g.splits - 1);
    if (lds.last) __hip_atomic_store(g.counters + seg, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!__builtin_amdgcn_readfirstlane(lds.last)) return;
  const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(g.parts + (size_t)seg * g.splits * kWideCols * (D + 8), (long long)g.splits * kWideCols * (D + 8) * 4);
  for (int c = tid >> 4; c < cols; c += kWideThreads / 16) {
    float mm = kNegInf, ll = 0.f, acc[NB][8];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[nb][e] = 0.f;
#pragma unroll 4
    for (int w = 0; w < g.splits; ++w) {
      const int at = ((w * kWideCols + c) * (D + 8)) * 4;
      const u32x2 ml = __builtin_amdgcn_raw_buffer_load_b64(rs, at + D * 4, 0, kSC1);
      const uint32_t mw = ml[0], lw = ml[1];
      const float pm = __builtin_bit_cast(float, mw), pl = __builtin_bit_cast(float, lw);
      const float m2 = fmaxf(mm, pm), u2 = m2 == kNegInf ? 0.f : m2;
      const float fa = __builtin_amdgcn_exp2f(mm - u2), fb = __builtin_amdgcn_exp2f(pm - u2);
      mm = m2;
      ll = ll * fa + pl * fb;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const u32x4 p0 = __builtin_amdgcn_raw_buffer_load_b128(rs, at + (nb * 128 + 8 * i) * 4, 0, kSC1);
        const u32x4 p1 = __builtin_amdgcn_raw_buffer_load_b128(rs, at + (nb * 128 + 8 * i + 4) * 4, 0, kSC1);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          acc[nb][e] = acc[nb][e] * fa + __builtin_bit_cast(float, (uint32_t)(e < 4 ? p0[e & 3] : p1[e & 3])) * fb;
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) write_block<BF>(g, q, head, column_at(g, from, c), nb, acc[nb], mm, ll);
  }
}

// Segments (column tiles of 64 times heads), at most.
long long wide_segments(const trellis_kv4_cache &c, const trellis_kv4_batch &b, int n_q_heads) {
  // (each sequence's last column tile may be partly filled)
  const long long tiles = ((long long)b.rows * (n_q_heads / c.n_kv_heads) + kWideCols - 1) / kWideCols + b.n_seq - 1;
  return (tiles > 1 ? tiles : 1) * c.n_kv_heads;
}

// Workgroups that share a segment's keys: where there are too few segments to fill the card, as
// many as do, but with no fewer than four tiles each of the longest context that the tables hold, and
// no more workgroups than the square root of its tiles, as one of them joins all their sums (one
// sequence, group 4, 8 heads; by this rule, without the root, without splitting: 16 rows over 30000
// tokens 53, 99, 220 us; 64 rows over 32000 78, 94, 754; over 4096 30, 27, 102; 256 rows over 8000
// 68, 68, 193).  Segments that fill the card, but not one and a half times, are halved: their last
// workgroups would run on alone (16 sequences of 3000 .. 6000 tokens, 40 rows each 133 -> 98 us, 48 rows
// 135 -> 103; 64 rows of 8 sequences and heads of 256 104 -> 99).
int wide_splits(const trellis_kv4_cache &c, const trellis_kv4_batch &b, int n_q_heads) {
  const long long segs = wide_segments(c, b, n_q_heads), room = (long long)micro_cus() * (c.head_dim == 128 ? wide_waves<1>() : wide_waves<2>());
  const long long tiles = ((long long)b.max_pages * c.page_size + kTile - 1) / kTile;
  long long n = room / segs;
  if (n == 1 && 2 * segs < 3 * room) n = 2;
  if (n > tiles / 4) n = tiles / 4;
  long long root = 1;
  while (root * root < tiles) ++root;
  if (n > root) n = root;
  return n < 1 ? 1 : n > 64 ? 64 : (int)n;
}

template <bool BF, int NB>
hipError_t launch(const AttnArgs &g, unsigned grid, hipStream_t stream) {
  const size_t lds = sizeof(WideLds<NB>);
  const auto kernel = kv4_attn_wide_kernel<BF, NB>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<grid, kWideThreads, lds, stream>>>(g);
  return hipGetLastError();
}

}  // namespace

size_t kv4_attn_wide_parts(const trellis_kv4_cache &c, const trellis_kv4_batch &b, int n_q_heads) {
  const int n = wide_splits(c, b, n_q_heads);
  return n == 1 ? 0 : (size_t)wide_segments(c, b, n_q_heads) * n * kWideCols * (c.head_dim + 8) * 4;
}

hipError_t launch_kv4_attn_wide(const AttnArgs &args, hipStream_t stream) {
  AttnArgs g = args;
  g.splits = wide_splits(g.a.c, g.a.b, g.a.n_q_heads);
  const unsigned grid = (unsigned)(wide_segments(g.a.c, g.a.b, g.a.n_q_heads) * g.splits);
  const bool bf = g.a.dtype == TRELLIS_KV4_BF16;
  if (g.a.c.head_dim == 128) return bf ? launch<true, 1>(g, grid, stream) : launch<false, 1>(g, grid, stream);
  return bf ? launch<true, 2>(g, grid, stream) : launch<false, 2>(g, grid, stream);
}

}  // namespace trellis
