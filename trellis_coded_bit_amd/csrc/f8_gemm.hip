// Products of block-scaled E4M3 rows with block-scaled E4M3 matrices, one or one per expert
// (include/trellis_f8.h).
//
// y[m][o] = sum over blocks b of 128 inputs of s[m][b] sw[o / 128][b] (q[m] . w[o] over the block):
// one v_mfma_f32_16x16x128_f8f6f4 forms a 16 x 16 tile of a block's products from zero, and a
// vector fma adds it times its scales.  Matrix rows are the tile's rows and tokens its columns, so
// a lane's four sums belong to one token and take one factor.  The scales are not put into the
// instruction's own: those are powers of two.
//
// Rounding: the instruction adds the products of eight neighbouring channels in steps of 2^-13 of the
// power of two of the largest one's factors, cut off towards zero, and the eights in about 24 bits
// (measured; the form without scales does the same), which leaves a block's sum off by 2e-5 rms.
// All else is f32, rounded once to 16 bits at the end.
#include <climits>
#include <cmath>

#include "f8_device.h"
#include "f8_tiles.h"

namespace trellis {

namespace {

typedef int intx8 __attribute__((ext_vector_type(8)));

constexpr int kLds = 163840;  // bytes of shared memory of a CU

struct GemmArgs {
  F8Gemm g;
  uint32_t *errword;
  int kb;         // blocks of 128 inputs
  int col_tiles;  // tiles over out_features
  int row_tiles;  // tiles over rows, at most
  int tile_rows;  // rows of a tile, at most
  int y8, y16;    // every row of y begins at a multiple of 8, 16 bytes
  int splits;     // of a tile's blocks among workgroups (many rows of one matrix)
  float *parts;   // splits > 1: their sums, [splits][rows][part_row]
  int64_t part_row;
};

template <int U>
__device__ __forceinline__ RowTiles find_tiles(const GemmArgs &p, int at, bool report) {
  return row_tiles_at<U>(p.g.offsets, p.g.L.n_experts, p.g.rows, p.tile_rows, at, report ? p.errword : nullptr);
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

// ---------------------------------------------------------------------------------------
// Rows of 128 bytes through shared memory, in both kernels: a copy takes eight of them, 1 KB, past
// the registers.  Read straight into the products' registers, neighbouring lanes would have
// different rows and each take a turn of its own at the cache (one token over 17408 x 5120: 21 us).
// A row's eight chunks of 16 bytes are permuted, chunk p of row r holding the row's chunk
// p ^ (r & 7), so that the products' reads of one chunk from eight rows fall on eight places.
// ---------------------------------------------------------------------------------------

typedef __attribute__((address_space(1))) const void gbl_void;
typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes a lane, copied to 16 * lane behind a place in shared memory, past the registers.
__device__ __forceinline__ void copy16(const void *from, void *to) {
  __builtin_amdgcn_global_load_lds((gbl_void *)from, (lds_void *)to, 16, 0, 0);
}
__device__ __forceinline__ void copy4(const void *from, void *to) {
  __builtin_amdgcn_global_load_lds((gbl_void *)from, (lds_void *)to, 4, 0, 0);
}

// Lane l of a copy has row l / 8 of its eight; its chunk of block b.  Chunks behind in_features
// repeat the row's last one; the products take zeros of the matrix there.
__device__ __forceinline__ uint32_t copy_chunk(int lane, int b, int K) {
  return (uint32_t)min(8 * b + ((lane & 7) ^ (lane >> 3)), K / 16 - 1);
}

__device__ __forceinline__ intx8 operand(const char *row, int lane) {
  const int g = lane >> 4, r = lane & 7;
  const u32x4 a = *reinterpret_cast<const u32x4 *>(row + ((g ^ r) << 4));
  const u32x4 b = *reinterpret_cast<const u32x4 *>(row + (((g + 4) ^ r) << 4));
  return intx8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}
// The chunks behind `rest` channels of a block become zero.
__device__ __forceinline__ void clear_behind(intx8 &w, int lane, int rest) {
  const int g = lane >> 4;
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = 16 * (g + 4 * (j >> 2)) < rest ? w[j] : 0;
}

// Whether one of a wave's sums is infinite or not a number (which a maximum is if an operand is).
template <int MF, int NT>
__device__ __forceinline__ bool any_far(const floatx4 (&acc)[MF][NT]) {
  float top = 0.f;
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        top = __builtin_elementwise_maximum(__builtin_elementwise_maximum(fabsf(acc[m][n][j]), fabsf(acc[m][n][j + 1])), top);
  return __any(!(top < INFINITY));
}

// Whether a row's and the matrix's scale of one of a wave's blocks are numbers whose product is none in f32.
template <int MF>
__device__ __forceinline__ bool far_scales(const GemmArgs &p, const float *sw, const int (&src)[MF], int first, int step, int end) {
  bool far = false;
#pragma clang loop unroll(disable)
  for (int b = first + step * ((int)(opaque_tid() & 63) >> 4); b < end; b += 4 * step) {  // (16 rows a tile, a quarter of the blocks a lane)
    const float t = ldg(sw + b);
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      const float s = ldg(p.g.s + (int64_t)src[m] * p.g.s_row + b);
      far |= fabsf(s) < INFINITY && fabsf(t) < INFINITY && !(fabsf(s * t) < INFINITY);
    }
  }
  return __any(far);
}

// A wave's sums again, for what the kernels' loops do not: they multiply a block's two scales first,
// and where that leaves f32 the block's sum may be zero or small and the result finite.  There the sum
// meets one scale after the other (both are above 1, so the first product is infinite only if the
// result is); every other block gives the same bits as in the loops.  w: the tile's first matrix row, n0;
// row: the lane's first behind it; sw: the matrix's scales; src: rows of q; blocks first, first + step
// ..., below end.  Done only where sums are not finite and the scales ask for it: the test of the sums
// costs the wide kernel up to 0.3 % (experts' tiles; 1.2 % by a comparison for each sum), and a row that
// stands for NaN no more than its noise (2048 x 17408 x 5120; 505 us for the 209 without the look at the scales).
template <int MF, int NT>
__device__ __forceinline__ void sums_again(const GemmArgs &p, const char *w, int n0, int row, const float *sw, const int (&src)[MF],
                                           int first, int step, int end, floatx4 (&acc)[MF][NT]) {
  const int K = p.g.L.in_features, lane = opaque_tid() & 63, g = lane >> 4;
  auto load = [&](const char *at, int b) {
    const int c = 8 * b + g, last = K / 16 - 1;
    const u32x4 x = ldg(reinterpret_cast<const u32x4 *>(at + 16 * min(c, last))), y = ldg(reinterpret_cast<const u32x4 *>(at + 16 * min(c + 4, last)));
    return intx8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  };
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma clang loop unroll(disable)
  for (int b = first; b < end; b += step) {
    const float t = ldg(sw + b);
    intx8 a[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      a[n] = load(w + (int64_t)min(row + 16 * n, p.g.L.out_features - 1 - n0) * K, b);
      clear_behind(a[n], lane, K - 128 * b);
    }
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      const intx8 x = load(reinterpret_cast<const char *>(p.g.q) + (int64_t)src[m] * p.g.q_row, b);
      const float s = ldg(p.g.s + (int64_t)src[m] * p.g.s_row + b), f = s * t;
      const bool far = !(fabsf(f) < INFINITY);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
        const floatx4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[n], x, zero, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][n][j] = fmaf(far ? d[j] * s : d[j], far ? t : f, acc[m][n][j]);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// Few rows: the matrix streams through once, and its bytes bound the kernel.
// ---------------------------------------------------------------------------------------

// A wave's place for one block: 16 NT matrix rows and their scale, 8 XC tokens.
template <int XC, int NT>
struct NarrowStage {
  static constexpr int copies = 2 * NT + XC + 1;
  alignas(16) char w[NT * 2048], x[XC * 1024];
  float sw[64];
};

// A wave's places, and its tokens' scales for eight blocks, two eights in turn: [token][block], a copy
// eight tokens.  (One block's scales are a line a token, as many as its codes: 37 rows by 5120 x 6144
// took 13.4 us so and take 12.6, 64 rows 17.5 and 15.3, in no cache.)
template <int XC, int NT, int D>
struct NarrowWave {
  NarrowStage<XC, NT> ring[D];
  float sx[2][XC * 64];
};

// A workgroup takes 16 NT matrix rows by 8 XC tokens; its waves take the blocks in turn, and their sums
// are added in the order of the waves.  `reps` tiles of matrix rows follow each other.  A wave copies
// into D places of its own, D - 1 blocks ahead over all its tiles, and needs no other wave for that;
// behind the last it copies that one again, so that the number of copies under way is a constant.
// One token over 17408 x 5120 takes 15.4 us (5.8 TB/s of the 6.4 that a stream reads at; 18 where the
// matrix is in no cache), 37 tokens over 5120 x 6144 9.6 (tokens in sixteens: 10.7), 33 tokens' 264
// entries over 256 experts' 4096 x 6144 605 to 645.  With more tokens it is far from the matrix's bytes,
// and what bounds it is not shown.  Of 64 tokens by 5120 x 6144, 15.7 us in no cache, a copy of the kernel
// that reads the same few token lines takes 11.8, the bytes alone 5; five or six waves in flight instead
// of four take no less.  Nor is it the CUs without a workgroup: 37 tokens by 2560, 5120, 8192 and 10240 x
// 6144 (80, 160, 256 and 320 workgroups) take 9.6, 12.8, 21.4 and 23.7 us in no cache, the matrix's
// and the tokens' copies together 5 to 6 TB/s from 160 workgroups on.
template <bool BF, int XC, int NT, int D>
__global__ __launch_bounds__(512) void narrow_kernel(GemmArgs p, int reps, int whole, int rest) {
  using Stage = NarrowStage<XC, NT>;
  using Wave = NarrowWave<XC, NT, D>;
  constexpr int MF = (XC + 1) / 2;  // tiles of 16 tokens (of an odd XC the last has its eight twice)
  extern __shared__ char raw[];
  const trellis_f8_linear &L = p.g.L;
  const int K = L.in_features, N = L.out_features, nb = (N + 127) / 128, kb = p.kb;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int i = lane & 15;
  Wave &mine = reinterpret_cast<Wave *>(raw)[wave];
  floatx4 *sums = reinterpret_cast<floatx4 *>(raw + waves * sizeof(Wave));  // [waves][MF][NT][64]
  const int groups = (p.col_tiles + reps - 1) / reps;
  const int rt = blockIdx.x / groups, c0 = (blockIdx.x - rt * groups) * reps, c1 = min(c0 + reps, p.col_tiles);
  const bool checks = rt == p.row_tiles;  // (the last of a grouped call: the offsets, to their end)
  const RowTiles tiles = find_tiles<8>(p, checks ? INT_MAX : rt, checks);
  if (tiles.e < 0) return;
  const RowTile t = tiles[rt - tiles.first];
  int src[XC];  // rows of q of the lane's tokens
  uint32_t xat[XC];  // and where they begin, in 16 bytes
#pragma unroll
  for (int j = 0; j < XC; ++j) {
    src[j] = max(source_row(p, min(t.row + 8 * j + (lane >> 3), t.end - 1)), 0);
    xat[j] = (uint32_t)((uint64_t)src[j] * (uint64_t)(p.g.q_row >> 4));
  }
  const int turns = whole + (wave < rest), all = turns * (c1 - c0);  // of this wave: a tile's, all tiles'
  int turn = 0;
  auto copy_scales = [&](int eight) {
    // (after a tile's last turn its first one follows again, for the next tile)
    const int of = 8 * eight + (lane & 7), u = reps == 1 ? min(of, turns - 1) : of % turns;
#pragma unroll
    for (int j = 0; j < XC; ++j)
      copy4(p.g.s + (int64_t)src[j] * p.g.s_row + wave + waves * u, mine.sx[eight & 1] + 64 * j);
  };
  // what is copied next
  int ct = c0, cb = wave, slot = 0;
  const char *w;
  const float *sw;
  uint32_t wat[2 * NT];  // of the lane's matrix rows behind w, in 16 bytes
  auto aim = [&]() {
    const int n0 = ct * 16 * NT;
    w = reinterpret_cast<const char *>(L.w) + ((int64_t)t.e * N + n0) * K;
    sw = L.scale + ((int64_t)t.e * nb + (n0 >> 7)) * kb;
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) wat[j] = (uint32_t)min(8 * j + (lane >> 3), N - 1 - n0) * (uint32_t)(K >> 4);
  };
  auto copy = [&]() {
    const int b = min(cb, kb - 1);
    const uint32_t u = copy_chunk(lane, b, K);
    Stage &o = mine.ring[slot];
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) copy16(w + ((uint64_t)(wat[j] + u) << 4), o.w + 1024 * j);
#pragma unroll
    for (int j = 0; j < XC; ++j) copy16(p.g.q + ((uint64_t)(xat[j] + u) << 4), o.x + 1024 * j);
    copy4(sw + b, o.sw);
    slot = slot + 1 == D ? 0 : slot + 1;
    cb += waves;
    if (cb >= kb && ct + 1 < c1) {
      ++ct;
      cb = wave;
      aim();
    }
  };
  aim();
  copy();
  copy_scales(0);  // (arrived with the first block)
#pragma unroll
  for (int d = 1; d + 1 < D; ++d) copy();
  int now = 0;
  for (int c = c0; c < c1; ++c) {
    const int n0 = c * 16 * NT;
    floatx4 acc[MF][NT];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma clang loop unroll(disable)
    for (int b = wave; b < kb; b += waves) {
      copy();
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 1) * Stage::copies) : "memory");
      if ((turn & 7) == 4 && turn + 4 < all) copy_scales((turn >> 3) + 1);
      const float *sx = mine.sx[(turn >> 3) & 1] + (turn & 7);
      ++turn;
      const Stage &o = mine.ring[now];
      now = now + 1 == D ? 0 : now + 1;
      intx8 a[NT], x[MF];
      float f[MF];
#pragma unroll
      for (int n = 0; n < NT; ++n) a[n] = operand(o.w + (16 * n + i) * 128, lane);
#pragma unroll
      for (int m = 0; m < MF; ++m) x[m] = operand(o.x + (16 * m + (2 * m + 1 < XC ? i : i & 7)) * 128, lane);
#pragma unroll
      for (int m = 0; m < MF; ++m) f[m] = sx[128 * m + 8 * (2 * m + 1 < XC ? i : i & 7)] * o.sw[0];
      if (K - 128 * b < 128)
#pragma unroll
        for (int n = 0; n < NT; ++n) clear_behind(a[n], lane, K - 128 * b);
#pragma unroll
      for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
          const floatx4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[n], x[m], zero, 0, 0, 0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][n][j] = fmaf(d[j], f[m], acc[m][n][j]);
        }
      asm volatile("" ::: "memory");  // (the place's reads are done before its next copies)
    }
    if (any_far(acc)) {
      int rows[MF];
#pragma unroll
      for (int m = 0; m < MF; ++m) rows[m] = max(source_row(p, min(t.row + 16 * m + (2 * m + 1 < XC ? i : i & 7), t.end - 1)), 0);
      const float *scales = L.scale + ((int64_t)t.e * nb + (n0 >> 7)) * kb;
      if (far_scales(p, scales, rows, wave, waves, kb))
        sums_again<MF, NT>(p, reinterpret_cast<const char *>(L.w) + ((int64_t)t.e * N + n0) * K, n0, i, scales, rows, wave, waves, kb, acc);
    }
    __builtin_amdgcn_s_barrier();  // (the sums of the tile before have been read)
    asm volatile("" ::: "memory");
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) sums[((wave * MF + m) * NT + n) * 64 + lane] = acc[m][n];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    // a thread has four columns of one token
    for (int at = threadIdx.x; at < MF * NT * 64; at += blockDim.x) {
      floatx4 v = sums[at];
      for (int u = 1; u < waves; ++u) {
        const floatx4 o = sums[u * MF * NT * 64 + at];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += o[j];
      }
      const int l = at & 63, n = (at >> 6) % NT, m = (at >> 6) / NT;
      const int row = t.row + 16 * m + (l & 15), col = n0 + 16 * n + 4 * (l >> 4);
      if (row >= t.end) continue;
      const bool zero = p.g.order && source_row(p, row) < 0;
      uint16_t *y = p.g.y + (int64_t)row * p.g.y_row + col;
      uint16_t r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = f8_narrow<BF>(zero ? 0.f : v[j]);
      if (p.y8 && col + 4 <= N) {
        stg(reinterpret_cast<u32x2 *>(y), u32x2{r[0] | (uint32_t)r[1] << 16, r[2] | (uint32_t)r[3] << 16});
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < N) stg(y + j, r[j]);
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (no copy is under way when the shared memory goes to another workgroup)
}

template <bool BF, int XC, int NT, int D>
hipError_t launch_narrow(GemmArgs p, hipStream_t stream) {
  const trellis_f8_linear &L = p.g.L;
  p.tile_rows = 8 * XC;
  p.col_tiles = (L.out_features + 16 * NT - 1) / (16 * NT);
  p.row_tiles = p.g.offsets ? p.g.rows / p.tile_rows + min(p.g.rows, L.n_experts) : (p.g.rows + p.tile_rows - 1) / p.tile_rows;
  const long long tiles = (long long)p.row_tiles * p.col_tiles;
  // (in long calls a workgroup's first copies and its look at the offsets serve four tiles: a decode
  // batch's experts 678 -> 632 us.  Two rows an expert, us with one | four: 64 experts' 1024 x 6144, 2560
  // tiles, 72 | 73, 64 of 2048 x 6144, 5120 tiles, 138 | 141, 128 of 2048 x 4096, 10240 tiles, 201 | 182, 256 of
  // 1024 x 2048, as many, 116 | 92)
  const int reps = tiles > (1 << 24) ? (int)min((tiles + (1 << 22) - 1) >> 22, (long long)p.col_tiles) : tiles > 4096 ? 4 : 1;
  constexpr int each = (int)sizeof(NarrowWave<XC, NT, D>) + (XC + 1) / 2 * NT * 1024, most = (8 * each <= kLds ? 8 : 4) * each;
  static_assert(most <= kLds, "four waves fit");
  // (few tiles: 4 tokens by 256 x 16384 9.4 us with four waves, 7.5 with eight, 1 by 2048 x 8192 6.9 and
  // 6.2; elsewhere within 0.6)
  int waves = tiles < 256 && most == 8 * each ? 8 : 4;
  if (waves > p.kb) waves = p.kb;
  const long long grid = (long long)p.row_tiles * ((p.col_tiles + reps - 1) / reps) + (p.g.offsets ? 1 : 0);
  const int lds = waves * each;
  if (lds > 65536) {
    // (the most of any call: another thread's may be between this and its launch)
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(narrow_kernel<BF, XC, NT, D>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != hipSuccess) return e;
  }
  narrow_kernel<BF, XC, NT, D><<<(unsigned)grid, 64 * waves, lds, stream>>>(p, reps, p.kb / waves, p.kb % waves);
  return hipGetLastError();
}

// `each`: rows of a matrix, about.
template <bool BF>
hipError_t launch_few(const GemmArgs &p, long long each, hipStream_t stream) {
  int xc = each <= 64 ? (int)(each + 7) / 8 : 8;
  const long long cols = (p.g.L.out_features + 31) / 32;
  // Fewer tokens a workgroup where that gives less than a workgroup to half of the CUs (64 x 256 x 16384:
  // 18.1 -> 8.2 us, 64 x 1024 x 16384: 18.0 -> 9.0); up to 192 it costs as often as it gives (33 x 5120 x
  // 6144: 8.5 -> 12.2, 48 x 4096 x 6144: 9.8 -> 7.8).
  while (!p.g.offsets && xc > 1 && (p.g.rows + 8 * xc - 1) / (8 * xc) * cols < 128) xc = (xc + 1) / 2;
  // Two tiles of matrix rows a workgroup share what is read of the tokens.  Where that is little, one
  // tile each, unless two come to a workgroup a CU or the tiles are many (us of one | two, in a graph,
  // matrices in no cache: 1 row by 512 x 8192 5.5 | 6.3, 2048 x 8192 6.2 | 7.9, 9216 x 5120 12.2 | 13.7,
  // 17408 x 5120 18.2 | 19.9, 69632 x 5120 65 | 59; 16 rows by 2048 x 8192 7.3 | 8.6, 5120 x 5120 11.1 |
  // 9.7, 8192 x 5120 11.8 | 10.5, 9216 x 5120 14.8 | 16.6, 69632 x 5120 87 | 79).
  const long long two = (p.g.rows + 15) / 16 * cols;
  const bool one = xc <= 2 && two < 1024 && (two < 128 || two > 256);
  switch (xc) {
    case 1: return one ? launch_narrow<BF, 1, 1, 3>(p, stream) : launch_narrow<BF, 1, 2, 3>(p, stream);
    case 2: return one ? launch_narrow<BF, 2, 1, 3>(p, stream) : launch_narrow<BF, 2, 2, 3>(p, stream);
    case 3: return launch_narrow<BF, 3, 2, 3>(p, stream);
    case 4: return launch_narrow<BF, 4, 2, 3>(p, stream);
    case 5: return launch_narrow<BF, 5, 2, 2>(p, stream);
    case 6: return launch_narrow<BF, 6, 2, 2>(p, stream);
    case 7: return launch_narrow<BF, 7, 2, 2>(p, stream);
    default: return launch_narrow<BF, 8, 2, 2>(p, stream);
  }
}

// ---------------------------------------------------------------------------------------
// Many rows: 256 matrix rows by up to 256 tokens a workgroup of eight waves, 64 by up to 128 a wave.
//
// A block of 128 inputs takes a workgroup 1.70 to 1.85 us at 256 tokens (2320 to 2530 TFLOP/s over the
// card).  Of copies of the kernel that leave something out, the one without copies from memory takes
// 1.40, without the meetings 1.37 then, without the reads of shared memory 1.30, with the matrix
// instructions alone 1.10 to 1.26.  So no single part bounds it: the matrix unit is busy 45 % of the
// time, and fmas (half as many cycles as the products), operand reads and copies (together half of
// shared memory's cycles, without conflicts) do not all fit beside it with two waves a SIMD; a third
// would not have the registers for its sums, which vector instructions must reach.
// 2048 rows by 17408 x 5120: 186 to 190 us (1950 TFLOP/s; 680 tiles of up to 224 tokens, 2.66 turns in
// the time of 3).  64 experts' 32768 rows by 4096 x 6144: 910 to 940 us (1790).
// ---------------------------------------------------------------------------------------

constexpr int kWideThreads = 512, kWideOut = 256, kWideRows = 256;

struct WideLds {
  alignas(16) char w[2][kWideOut * 128], x[2][kWideRows * 128];  // a block of 128 inputs, two in turn
  alignas(16) float sx[2][kWideRows], sw[2][64];
};

// Where a lane's copies come from.
struct WideFrom {
  uint32_t w[4], x[4];  // rows 64 j + 8 wave + l / 8: in 16 bytes from the tile's first row, from q
  const float *s;       // waves 0..3: the scales of row 64 wave + l; 4..7: of the tile's matrix blocks
  int chunk;
};

// The copies of a block are made in two parts: the matrix and the tokens that the first products
// take, and the other tokens (64 a copy: what two of a wave's tiles take) with the scales.
template <int MF>
struct WidePart {
  static constexpr int copies = (MF + 1) / 2, first = copies / 2, second = copies - first + 1;
  static constexpr int tiles = 2 * first;  // of a wave in the first part
};
__device__ __forceinline__ void wide_copy_x(const GemmArgs &p, const WideFrom &f, int wave, uint32_t u, int j, WideLds &lds, int buf) {
  // (of an odd number of tiles the last copy's second half would not be read; it is made all the
  // same, so that every wave has the same number under way)
  copy16(p.g.q + ((uint64_t)(f.x[j] + u) << 4), lds.x[buf] + (64 * j + 8 * wave) * 128);
}
template <int MF>
__device__ __forceinline__ void wide_copy1(const GemmArgs &p, const char *w, const WideFrom &f, int wave, int b, WideLds &lds) {
  const uint32_t u = (uint32_t)min(8 * b + f.chunk, p.g.L.in_features / 16 - 1);
  const int buf = b & 1;
#pragma unroll
  for (int j = 0; j < 4; ++j) copy16(w + ((uint64_t)(f.w[j] + u) << 4), lds.w[buf] + (64 * j + 8 * wave) * 128);
#pragma unroll
  for (int j = 0; j < WidePart<MF>::first; ++j) wide_copy_x(p, f, wave, u, j, lds, buf);
}
template <int MF>
__device__ __forceinline__ void wide_copy2(const GemmArgs &p, const WideFrom &f, int wave, int b, WideLds &lds) {
  const uint32_t u = (uint32_t)min(8 * b + f.chunk, p.g.L.in_features / 16 - 1);
#pragma unroll
  for (int j = WidePart<MF>::first; j < WidePart<MF>::copies; ++j) wide_copy_x(p, f, wave, u, j, lds, b & 1);
  copy4(f.s + b, wave < 4 ? lds.sx[b & 1] + 64 * wave : lds.sw[b & 1]);  // (waves 4..7: the same)
}

// Waits until at most N of this wave's copies are under way, then for the workgroup's other waves.
// Reads of shared memory stay on their side of it.
template <int N>
__device__ __forceinline__ void wide_meet() {
  static_assert(N < 16, "the lower four bits of the count");
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// A wave's 64 matrix rows by 16 MF tokens over all blocks.  Its tile m takes tokens 32 m + 16 wm ..
// A product's results are added to the sums while the next ones run, and operands are read one tile
// ahead, the next block's first ones too: what they wait for was met half a block before.  On entry
// blocks 0 and 1 are in shared memory.  Two meetings a block: at the middle all waves have read the
// block's matrix and first tokens, whose places then take the block after next; at the end the rest.
// (One meeting a block, results used at once and operands read within a block: 219 us for the 195 that
// this gave 2048 x 17408 x 5120.)
constexpr int kBehind = 3;  // products between one and the use of its results (at most 4)

template <int MF>
__device__ __forceinline__ void wide_blocks(const GemmArgs &p, const char *from_w, const WideFrom &f, int wave, WideLds &lds,
                                            int kb, int rest, floatx4 (&acc)[MF][4]) {
  const int lane = opaque_tid() & 63;
  using Part = WidePart<MF>;
  const int i = lane & 15, wm = wave & 1, wn = wave >> 1;
  const char *wp = lds.w[0] + (64 * wn + i) * 128, *xp = lds.x[0] + (16 * wm + i) * 128;
  constexpr int kBuf = kWideOut * 128;
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int n = 0; n < 4; ++n) acc[m][n] = floatx4{0.f, 0.f, 0.f, 0.f};
  intx8 w[4], next;
#pragma unroll
  for (int n = 0; n < 4; ++n) w[n] = operand(wp + n * 2048, lane);
  next = operand(xp, lane);
  const float *sx = lds.sx[0] + 16 * wm + i;
  float s[2] = {0.f, 0.f};              // of this tile's products and the last one's
  floatx4 d[kBehind];                   // the last products
#pragma unroll
  for (int k = 0; k < kBehind; ++k) d[k] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma clang loop unroll(disable)
  for (int b = 0; b < kb; ++b) {
    const int buf = b & 1;
    if (rest && b == kb - 1)
#pragma unroll
      for (int n = 0; n < 4; ++n) clear_behind(w[n], lane, rest);
    const float sw = lds.sw[buf][wn >> 1];
    float sn = sx[buf * kWideRows];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      if (m == Part::tiles) {
        // (before the block's first product its matrix operands may still be on their way from
        // where the copies go)
        if (m == 0) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wide_meet<Part::second>();
        if (b + 2 < kb) wide_copy1<MF>(p, from_w, f, wave, b + 2, lds);
      }
      const intx8 x = next;
      if (m + 1 < MF) next = operand(xp + buf * kBuf + (m + 1) * 4096, lane);
      else if (Part::tiles) next = operand(xp + (buf ^ 1) * kBuf, lane);
      s[1] = s[0];
      s[0] = sn * sw;
      if (m + 1 < MF) sn = sx[buf * kWideRows + 32 * (m + 1)];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
        const floatx4 e = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[n], x, zero, 0, 0, 0, 0, 0, 0);
        floatx4 &into = acc[n < kBehind ? (m + MF - 1) % MF : m][(n + 4 - kBehind) & 3];
        const float by = s[n < kBehind];
#pragma unroll
        for (int j = 0; j < 4; ++j) into[j] = fmaf(d[0][j], by, into[j]);
        asm volatile("" : "+v"(into));  // (here, not where the sums are used)
#pragma unroll
        for (int k = 0; k + 1 < kBehind; ++k) d[k] = d[k + 1];
        d[kBehind - 1] = e;
        if (m + 1 == MF) w[n] = operand(wp + (buf ^ 1) * kBuf + n * 2048, lane);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (b + 2 < kb) {
      wide_meet<4 + Part::first>();
      wide_copy2<MF>(p, f, wave, b + 2, lds);
    } else {
      wide_meet<0>();
    }
    if (!Part::tiles) next = operand(xp + (buf ^ 1) * kBuf, lane);  // (all tokens are in the second part)
  }
#pragma unroll
  for (int n = 0; n < kBehind; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[MF - 1][n + 4 - kBehind][j] = fmaf(d[n][j], s[0], acc[MF - 1][n + 4 - kBehind][j]);
}

// A tile to be: its rows, its first matrix row, its blocks, and where its copies come from.
struct WideTile {
  RowTile t;
  int n0, split, kb, rest;  // rest: channels of a last, partial block
  const char *w;
  WideFrom f;
};

// Looks a tile up and starts the copies of its first two blocks.
__device__ __forceinline__ void wide_begin(const GemmArgs &p, WideTile &x, int wave, WideLds &lds) {
  const int lane = opaque_tid() & 63;
  const trellis_f8_linear &L = p.g.L;
  const int K = L.in_features, N = L.out_features, nb = (N + 127) / 128;
  x.w = reinterpret_cast<const char *>(L.w) + ((int64_t)x.t.e * N + x.n0) * K;
  WideFrom &f = x.f;
  const int each = (p.kb + p.splits - 1) / p.splits, b0 = x.split * each;
  x.kb = min(each, p.kb - b0);
  x.rest = b0 + x.kb == p.kb ? K & 127 : 0;
  f.chunk = 8 * b0 + ((lane & 7) ^ (lane >> 3));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 64 * j + 8 * wave + (lane >> 3);
    f.w[j] = (uint32_t)min(r, N - 1 - x.n0) * (uint32_t)(K >> 4);
    f.x[j] = (uint32_t)((uint64_t)max(source_row(p, min(x.t.row + r, x.t.end - 1)), 0) * (uint64_t)(p.g.q_row >> 4));
  }
  if (wave < 4) f.s = p.g.s + (int64_t)max(source_row(p, min(x.t.row + 64 * wave + lane, x.t.end - 1)), 0) * p.g.s_row;
  else f.s = L.scale + ((int64_t)x.t.e * nb + min((x.n0 >> 7) + (lane & 1), nb - 1)) * p.kb;
  f.s += b0;
  const int copies = (x.t.end - x.t.row + 63) >> 6;
  for (int b = 0; b < min(x.kb, 2); ++b) {
    const uint32_t u = (uint32_t)min(8 * b + f.chunk, K / 16 - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) copy16(x.w + ((uint64_t)(f.w[j] + u) << 4), lds.w[b] + (64 * j + 8 * wave) * 128);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < copies) wide_copy_x(p, f, wave, u, j, lds, b);
    copy4(f.s + b, wave < 4 ? lds.sx[b] + 64 * wave : lds.sw[b]);
  }
}

// The sums of a tile, rounded and stored, or as they are where others are to be added.  A lane has four
// neighbouring columns of one token in each of its tiles; two tiles' are exchanged between neighbouring
// rows of lanes so that it has eight of one.
template <bool BF, int MF>
__device__ __forceinline__ void wide_store(const GemmArgs &p, const RowTile &t, int n0, int split, int wave, const floatx4 (&acc)[MF][4]) {
  const int lane = opaque_tid() & 63;
  const int N = p.g.L.out_features, wm = wave & 1, wn = wave >> 1, g = lane >> 4;
  if (p.splits > 1) {
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      const int row = t.row + 32 * m + 16 * wm + (lane & 15);
      float *to = p.parts + ((int64_t)split * p.g.rows + row) * p.part_row;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int c = n0 + 64 * wn + 16 * n + 4 * g;
        if (row < t.end && c < N) stg(reinterpret_cast<floatx4 *>(to + c), acc[m][n]);
      }
    }
    return;
  }
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    const int row = t.row + 32 * m + 16 * wm + (lane & 15);
    const bool live = row < t.end;
    const bool zero = live && p.g.order && source_row(p, row) < 0;
    uint16_t *y = p.g.y + (int64_t)row * p.g.y_row;
#pragma unroll
    for (int n = 0; n < 4; n += 2) {
      u32x2 v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const floatx4 &a = acc[m][n + h];
          v[h][j] = zero ? 0u : f8_narrow<BF>(a[2 * j]) | (uint32_t)f8_narrow<BF>(a[2 * j + 1]) << 16;
        }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const auto r = __builtin_amdgcn_permlane16_swap(v[0][j], v[1][j], false, false);
        v[0][j] = r[0];
        v[1][j] = r[1];
      }
      // lanes of even rows have the first tile's columns, those of odd rows the second's
      const int c = n0 + 64 * wn + 16 * (n + (g & 1)) + 8 * (g >> 1);
      if (!live) continue;
      if (p.y16 && c + 8 <= N) {
        stg(reinterpret_cast<u32x4 *>(y + c), u32x4{v[0][0], v[0][1], v[1][0], v[1][1]});
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < N) stg(y + c + j, (uint16_t)(v[j >> 2][(j >> 1) & 1] >> (16 * (j & 1))));
      }
    }
  }
}

// Looks up what a workgroup does in its turn, and starts its first copies.  Tiles come in an order
// that keeps what runs at a time on one XCD (every eighth workgroup, with a run of the list) close
// together: expert after expert; of an expert up to eight row tiles by the column tiles, row tiles
// first, so that they share the matrix's rows while these are in the XCD's cache (the experts above:
// 26.0 M lines missed there, 35.5 M where eight row tiles were taken whatever their experts; 2 to 6 %).
__device__ __forceinline__ bool wide_next(const GemmArgs &p, int row_tiles, int turn, int wave, WideTile &x, WideLds &lds) {
  const int tiles = row_tiles * p.col_tiles, total = tiles * p.splits, per = total >> 3, rest = total & 7;
  // (a turn's tiles move on by one workgroup: a band's tall row tiles would be the same ones' every time)
  const int xcd = blockIdx.x & 7, n = (int)gridDim.x >> 3, i = turn * n + ((int)(blockIdx.x >> 3) + turn) % n;
  if (i >= per + (xcd < rest)) return false;
  int at = xcd * per + min(xcd, rest) + i;
  x.split = at / tiles;
  at -= x.split * tiles;
  const RowTiles r = find_tiles<32>(p, at / p.col_tiles, false);
  if (r.e < 0) return false;
  at -= r.first * p.col_tiles;
  const int bands = (r.tiles + 7) >> 3, band_rows = (r.tiles + bands - 1) / bands, band = at / (band_rows * p.col_tiles);
  at -= band * band_rows * p.col_tiles;
  const int high = min(band_rows, r.tiles - band * band_rows), ct = at / high;
  x.t = r[band * band_rows + at - ct * high];
  x.n0 = ct * kWideOut;
  wide_begin(p, x, wave, lds);
  return true;
}

// One tile's products; the next tile's first copies are under way while this one is stored.
template <bool BF, int MF>
__device__ __forceinline__ bool wide_tile(const GemmArgs &p, int row_tiles, int turn, int wave, WideTile &x, WideLds &lds) {
  floatx4 acc[MF][4];
  wide_blocks<MF>(p, x.w, x.f, wave, lds, x.kb, x.rest, acc);
  if (any_far(acc)) {
    const trellis_f8_linear &L = p.g.L;
    const int i = opaque_tid() & 15, wm = wave & 1, wn = wave >> 1, nb = (L.out_features + 127) / 128;
    const int b0 = x.split * ((p.kb + p.splits - 1) / p.splits);
    int rows[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m) rows[m] = max(source_row(p, min(x.t.row + 32 * m + 16 * wm + i, x.t.end - 1)), 0);
    const float *scales = L.scale + ((int64_t)x.t.e * nb + min((x.n0 >> 7) + (wn >> 1), nb - 1)) * p.kb;
    if (far_scales(p, scales, rows, b0, 1, b0 + x.kb)) sums_again<MF, 4>(p, x.w, x.n0, 64 * wn + i, scales, rows, b0, 1, b0 + x.kb, acc);
  }
  const RowTile t = x.t;
  const int n0 = x.n0, split = x.split;
  const bool more = wide_next(p, row_tiles, turn, wave, x, lds);
  wide_store<BF, MF>(p, t, n0, split, wave, acc);
  return more;
}

// One workgroup a CU, tile after tile.  The number of a tile's tokens, in 32s, picks the code for it.
template <bool BF>
__global__ __launch_bounds__(kWideThreads, 2) void wide_kernel(GemmArgs p) {
  extern __shared__ char raw[];
  WideLds &lds = *reinterpret_cast<WideLds *>(raw);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row_tiles = find_tiles<32>(p, INT_MAX, blockIdx.x == 0).first;
  WideTile x;
  bool more = wide_next(p, row_tiles, 0, wave, x, lds);
  for (int turn = 1; more; ++turn) {
    wide_meet<0>();
    switch ((x.t.end - x.t.row + 31) >> 5) {
      case 8: more = wide_tile<BF, 8>(p, row_tiles, turn, wave, x, lds); break;
      case 7: more = wide_tile<BF, 7>(p, row_tiles, turn, wave, x, lds); break;
      case 6: more = wide_tile<BF, 6>(p, row_tiles, turn, wave, x, lds); break;
      case 5: more = wide_tile<BF, 5>(p, row_tiles, turn, wave, x, lds); break;
      case 4: more = wide_tile<BF, 4>(p, row_tiles, turn, wave, x, lds); break;
      case 3: more = wide_tile<BF, 3>(p, row_tiles, turn, wave, x, lds); break;
      case 2: more = wide_tile<BF, 2>(p, row_tiles, turn, wave, x, lds); break;
      default: more = wide_tile<BF, 1>(p, row_tiles, turn, wave, x, lds); break;
    }
  }
}

// The splits' sums added in their order, rounded and stored: four columns a thread.
template <bool BF>
__global__ __launch_bounds__(256) void join_kernel(GemmArgs p) {
  const int N = p.g.L.out_features, quads = (N + 3) >> 2;
  const int64_t split = p.g.rows * p.part_row;
  for (uint32_t at = blockIdx.x * 256 + threadIdx.x; at < (uint32_t)p.g.rows * (uint32_t)quads; at += gridDim.x * 256) {
    const int row = (int)(at / (uint32_t)quads), c = 4 * (int)(at - (uint32_t)row * (uint32_t)quads);
    const float *from = p.parts + row * p.part_row + c;
    floatx4 v = ldg(reinterpret_cast<const floatx4 *>(from));
    for (int s = 1; s < p.splits; ++s) {
      const floatx4 o = ldg(reinterpret_cast<const floatx4 *>(from + s * split));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += o[j];
    }
    uint16_t *y = p.g.y + (int64_t)row * p.g.y_row + c, r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = f8_narrow<BF>(v[j]);
    if (p.y8 && c + 4 <= N) {
      stg(reinterpret_cast<u32x2 *>(y), u32x2{r[0] | (uint32_t)r[1] << 16, r[2] | (uint32_t)r[3] << 16});
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < N) stg(y + j, r[j]);
    }
  }
}

// How a call is divided.  Times in microseconds, as measured: the narrow kernel takes 0.86 ns for a
// block of 64 tokens by 32 matrix rows over the whole card; a wide workgroup 0.45 + 0.156 a block for
// every 32 of its tokens, and 3 a tile; a split's sums are written and read at 5 TB/s by one launch
// more.  Matrices in no cache, narrow | wide, blocks whole | wide, blocks shared: 5120 x 6144 with 32
// rows 12.0 | 56 | 18, 64 rows 15.7 | 57 | 20, 128 rows 23.3 | 57 | 23.4, 256 rows 35 | 57 | 31, 512 rows
// 58 | 56 | 40; 17408 x 5120 with 32 rows 30 | 54 | 30, 64 rows 40 | 55 | 33, 128 rows 56 | 53 | 40.
//
// Experts' wide tiles are priced as full ones (256 rows, 1.70 a block) although they run at the rows that
// they have, up to 32 rows an expert are not weighed, and rows whose expert is not here count as if it
// were.  So few rows an expert stay narrow longer than they should.  Narrow | wide with 16, 33, 48, 64 and
// 96 rows each, * what is taken: 64 experts of 2048 x 2048 68* | 60, 82* | 62, 90* | 64, 101* | 64, 159 |
// 71*; of 6144 x 2048 194* | 159, 235* | 167, 254* | 175, 281* | 181, 446 | 201*; of 4096 x 6144 317* | 301,
// 385 | 306*, 420 | 312*, 464 | 320*, 716 | 347*; 256 of 2048 x 2048 257* | 207, 314* | 220, 341* | 229,
// 381* | 236, 621 | 263*; 16 of 4096 x 6144 105* | 84, 121 | 86*, 132 | 87*, 146 | 89*, 182 | 96*.
struct Plan {
  bool narrow;
  int tile_rows, splits;
};
Plan plan(const trellis_f8_linear &L, int rows, bool grouped) {
  const long long kb = (L.in_features + 127) / 128, N = L.out_features, col_tiles = (N + kWideOut - 1) / kWideOut;
  const long long matrices = grouped ? min(rows, L.n_experts) : 1;
  const double each = (double)rows / matrices;
  Plan best{true, 0, 1};
  if (each <= 32) return best;
  double least = 4 + 0.86e-3 * (matrices * ceil(each / 64) * ((N + 31) / 32)) * kb;
  for (int mf = 8; mf >= 2; --mf) {
    const double tiles = matrices * ceil(each / (32 * mf)) * col_tiles, block = 0.45 + 0.156 * mf;
    for (int splits = 1; splits <= (grouped ? 1 : 16) && splits * 4 <= max(kb, 4LL); ++splits) {
      const long long part = (kb + splits - 1) / splits;
      if ((kb + part - 1) / part != splits) continue;  // (each split has blocks)
      const double time = ceil(tiles * splits / 256) * (part * block + 3) + 1 +
                          (splits > 1 ? 2 + splits * (double)rows * N * 8 / 5e6 : 0);
      if (time < least) {
        least = time;
        best = {false, 32 * mf, splits};
      }
      if (tiles * splits >= 256) break;
    }
    if (grouped) break;  // (experts' rows are cut evenly into as few tiles as they take)
  }
  return best;
}

int64_t part_row(int N) { return (N + 3) & ~3; }

}  // namespace

size_t f8_gemm_workspace_bytes(const trellis_f8_linear &L, int rows, bool grouped) {
  const Plan d = rows > 0 ? plan(L, rows, grouped) : Plan{true, 0, 1};
  return kWsReserved + (d.splits > 1 ? (size_t)d.splits * rows * part_row(L.out_features) * 4 : 0);
}

hipError_t launch_f8_gemm(const F8Gemm &a, void *ws, hipStream_t stream) {
  GemmArgs p{};
  p.g = a;
  p.errword = static_cast<uint32_t *>(ws);
  p.kb = (a.L.in_features + 127) / 128;
  p.y8 = a.y_row % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 8 == 0;
  p.y16 = a.y_row % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
  const Plan d = plan(a.L, a.rows, a.offsets != nullptr);
  if (d.narrow) {
    const long long matrices = a.offsets ? min(a.rows, a.L.n_experts) : 1, each = (a.rows + matrices - 1) / matrices;
    return a.bf16 ? launch_few<true>(p, each, stream) : launch_few<false>(p, each, stream);
  }
  p.col_tiles = (a.L.out_features + kWideOut - 1) / kWideOut;
  p.tile_rows = d.tile_rows;
  p.splits = d.splits;
  p.part_row = part_row(a.L.out_features);
  p.parts = reinterpret_cast<float *>(static_cast<char *>(ws) + kWsReserved);
  p.row_tiles = a.offsets ? a.rows / p.tile_rows + min(a.rows, a.L.n_experts) : (a.rows + p.tile_rows - 1) / p.tile_rows;
  // one workgroup a CU (its shared memory holds one), whole eights of them for the XCDs
  const long long units = (long long)p.row_tiles * p.col_tiles * p.splits, grid = (min(units, 256LL) + 7) & ~7LL;
  const void *kernel = a.bf16 ? reinterpret_cast<const void *>(wide_kernel<true>) : reinterpret_cast<const void *>(wide_kernel<false>);
  hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(WideLds));
  if (e != hipSuccess) return e;
  if (a.bf16) wide_kernel<true><<<(unsigned)grid, kWideThreads, sizeof(WideLds), stream>>>(p);
  else wide_kernel<false><<<(unsigned)grid, kWideThreads, sizeof(WideLds), stream>>>(p);
  e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const long long quads = (long long)a.rows * ((a.L.out_features + 3) / 4);
  const unsigned join = (unsigned)min((quads + 255) / 256, 1LL << 16);
  if (a.bf16) join_kernel<true><<<join, 256, 0, stream>>>(p);
  else join_kernel<false><<<join, 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace trellis
