// Which rows of a product a workgroup takes: rows sorted by expert, every expert's cut into tiles of its
// own.  Included behind what it uses (ldg, opaque_tid, f8_error).
#pragma once

namespace trellis {

// Which rows a tile has: of expert e, rows [row, end).  e < 0: none.
struct RowTile {
  int e, row, end;
};

// An expert's rows [row, end) in tiles of `size`, `first` tiles of earlier experts before them.
struct RowTiles {
  int e, row, end, size, tiles, first;
  __device__ __forceinline__ RowTile operator[](int i) const { return {e, row + i * size, min(end, row + (i + 1) * size)}; }
};

// n rows as tiles of at most T rows, T a multiple of U: as few as that takes, of the same size (a
// multiple of U) but for the last.
struct Cut {
  int tiles, size;
};
template <int U>
__device__ __forceinline__ Cut cut_rows(int n, int T) {
  const int tiles = (n + T - 1) / T;
  const int size = tiles ? ((n + tiles - 1) / tiles + U - 1) / U * U : U;
  return {(n + size - 1) / size, size};
}

// The expert of tile `at` of the list: every expert's rows in tiles of at most T, expert after expert.
// Behind the last (at = INT_MAX, say) e is -1 and `first` the number of tiles.  The list ends at the
// first pair of offsets that is out of order or out of range, which is reported where there is an
// errword.  offsets NULL: all rows are one matrix's.  Called by whole waves.
//
// What comes back is an expert below E and rows below `rows` whatever the offsets are, also if they
// change between two loads (written by another stream that the caller did not wait for): a lane's
// counts come from what it has loaded, and lanes behind the last offset load nothing.
template <int U>
__device__ __forceinline__ RowTiles row_tiles_at(const int32_t *offsets, int E, int rows, int T, int at, uint32_t *errword) {
  if (!offsets) {
    const Cut c = cut_rows<U>(rows, T);
    return {at < c.tiles ? 0 : -1, 0, rows, c.size, c.tiles, at < c.tiles ? 0 : c.tiles};
  }
  const int lane = opaque_tid() & 63;
  int passed = 0;
  bool wrong = __ballot(ldg(offsets) != 0) != 0;
  for (int e0 = 0; e0 < E && !wrong; e0 += 256) {
    // four neighbouring experts a lane, their tiles summed, then over the lanes
    const int e = e0 + 4 * lane;
    int o[5], sum = 0;
    Cut c[4];
    o[0] = e <= E ? ldg(offsets + e) : 0;
#pragma unroll
    for (int k = 1; k < 5; ++k) o[k] = e + k <= E ? ldg(offsets + e + k) : o[k - 1];
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      bad |= o[k] < 0 || o[k + 1] < o[k] || o[k + 1] > rows;
      c[k] = cut_rows<U>(bad ? 0 : o[k + 1] - o[k], T);
      sum += c[k].tiles;
    }
    const uint64_t bads = __ballot(bad);
    if (bads && lane > __builtin_ctzll(bads)) sum = 0;
    int s = sum;
    for (int d = 1; d < 64; d <<= 1) {
      const int t = __shfl_up(s, d, 64);
      if (lane >= d) s += t;
    }
    const uint64_t has = __ballot(at < passed + s);
    if (has) {
      const int l = __builtin_ctzll(has);
      int first = passed + s - sum;
      RowTiles r = {e, 0, 0, U, 0, first};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (at >= first && at - first < c[k].tiles) r = {e + k, o[k], o[k + 1], c[k].size, c[k].tiles, first};
        first += c[k].tiles;
      }
      return {__builtin_amdgcn_readlane(r.e, l),    __builtin_amdgcn_readlane(r.row, l),   __builtin_amdgcn_readlane(r.end, l),
              __builtin_amdgcn_readlane(r.size, l), __builtin_amdgcn_readlane(r.tiles, l), __builtin_amdgcn_readlane(r.first, l)};
    }
    passed += __builtin_amdgcn_readlane(s, 63);
    wrong = bads != 0;
  }
  if (wrong && errword && lane == 0) f8_error(errword);
  return {-1, 0, 0, U, 0, passed};
}

}  // namespace trellis
