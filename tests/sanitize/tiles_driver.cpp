// Host driver of csrc/f8_tiles.h: a wave's 64 lanes as coroutines that meet at ballots, shuffles and
// readlanes.  Lists of offsets, right ones, wrong ones, and ones that change between two of a wave's loads:
// right ones give every row once and in order, and whatever they are, what comes back lies within the
// experts and the rows.  Exit status 0 when every expectation holds.
#include <ucontext.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

using std::min;

#define __device__
#define __forceinline__ inline

static int g_fail = 0;
#define EXPECT(c)                                                                    \
  do {                                                                               \
    if (!(c)) {                                                                      \
      if (g_fail++ < 10) std::fprintf(stderr, "line %d: %s\n", __LINE__, #c);        \
    }                                                                                \
  } while (0)

// The wave.
constexpr int kLanes = 64;
static ucontext_t g_home, g_ctx[kLanes];
static std::vector<char> g_stack[kLanes];
static int g_lane, g_arrived, g_round, g_waits[kLanes];
static bool g_done[kLanes];
static uint64_t g_slot[2][kLanes];

static const uint64_t *meet(uint64_t v) {
  const int me = g_lane, round = g_round;
  g_slot[round & 1][me] = v;
  if (++g_arrived == kLanes) {
    g_arrived = 0;
    ++g_round;
  } else {
    g_waits[me] = round;
    swapcontext(&g_ctx[me], &g_home);
  }
  return g_slot[round & 1];
}
static uint64_t sim_ballot(bool b) {
  const uint64_t *s = meet(b);
  uint64_t r = 0;
  for (int l = 0; l < kLanes; ++l) r |= s[l] << l;
  return r;
}
static int sim_read(int v, int from) { return (int)meet((uint32_t)v)[from]; }
static int sim_up(int v, int d) {
  const int l = g_lane;
  return (int)meet((uint32_t)v)[l < d ? l : l - d];
}
#define __ballot(b) sim_ballot(b)
#define __shfl_up(v, d, w) sim_up(v, d)
#define __builtin_amdgcn_readlane(v, l) sim_read(v, l)

// Memory: the offsets, which change after a number of loads.
static std::vector<int32_t> g_offsets, g_later;
static long g_left;
static uint32_t g_error;

namespace trellis {
static int opaque_tid() { return g_lane; }
static int32_t ldg(const int32_t *p) {
  EXPECT(p >= g_offsets.data() && p < g_offsets.data() + g_offsets.size());
  if (g_left-- == 0) g_offsets = g_later;
  return *p;
}
static void f8_error(uint32_t *e) { *e |= 1; }
}  // namespace trellis

#include "../../trellis_coded_bit_amd/csrc/f8_tiles.h"

using trellis::RowTiles;

static RowTiles g_result[kLanes];
static int g_E, g_rows, g_T, g_at, g_unit;

static void lane_main() {
  const int me = g_lane;
  g_result[me] = g_unit == 8 ? trellis::row_tiles_at<8>(g_offsets.data(), g_E, g_rows, g_T, g_at, &g_error)
                             : trellis::row_tiles_at<32>(g_offsets.data(), g_E, g_rows, g_T, g_at, &g_error);
  g_done[me] = true;
}

static RowTiles look(int at) {
  g_at = at;
  g_arrived = 0;
  for (int l = 0; l < kLanes; ++l) {
    g_done[l] = false;
    g_waits[l] = -1;
    if (g_stack[l].empty()) g_stack[l].resize(1 << 16);
    getcontext(&g_ctx[l]);
    g_ctx[l].uc_stack.ss_sp = g_stack[l].data();
    g_ctx[l].uc_stack.ss_size = g_stack[l].size();
    g_ctx[l].uc_link = &g_home;
    makecontext(&g_ctx[l], lane_main, 0);
  }
  for (bool going = true; going;) {
    going = false;
    for (int l = 0; l < kLanes; ++l) {
      if (g_done[l] || g_waits[l] == g_round) continue;
      g_lane = l;
      swapcontext(&g_home, &g_ctx[l]);
      going = true;
    }
  }
  for (int l = 0; l < kLanes; ++l) EXPECT(g_done[l]);
  for (int l = 1; l < kLanes; ++l) EXPECT(g_result[l].e == g_result[0].e && g_result[l].first == g_result[0].first);
  return g_result[0];
}

static void within(const RowTiles &r, int at) {
  EXPECT(r.e >= -1 && r.e < g_E);
  if (r.e < 0) return;
  EXPECT(r.tiles > 0 && r.first >= 0 && at >= r.first && at - r.first < r.tiles);
  for (int i = 0; i < r.tiles; ++i) {
    const trellis::RowTile t = r[i];
    EXPECT(t.e == r.e && t.row >= 0 && t.row < t.end && t.end <= g_rows && t.end - t.row <= g_T);
  }
}

int main() {
  std::mt19937 g(7);
  auto below = [&](int n) { return (int)(g() % (unsigned)n); };
  for (int trial = 0; trial < 200; ++trial) {
    g_E = trial % 5 == 0 ? 1 + below(600) : 1 + below(40);
    g_unit = trial & 1 ? 8 : 32;
    g_T = g_unit * (1 + below(8));
    std::vector<int32_t> right(g_E + 1);
    for (int e = 0; e < g_E; ++e) right[e + 1] = right[e] + (below(3) ? below(2 * g_T) : 0);
    g_rows = right[g_E] + below(3);
    // the list itself: every row of every expert once
    g_offsets = g_later = right;
    g_left = -1;
    g_error = 0;
    int row = 0, e = -1;
    const int total = look(INT_MAX).first;
    EXPECT(g_error == 0);
    for (int at = 0; at < total; at += 1 + below(1 + total / 20)) {
      const RowTiles r = look(at);
      within(r, at);
      EXPECT(r.e >= 0 && r.row == right[r.e] && r.end == right[r.e + 1]);
      EXPECT(r[0].row == r.row && r[r.tiles - 1].end == r.end && (r.e > e ? r.row >= row : r.e == e));
      e = r.e;
      row = r.row;
    }
    EXPECT(look(total).e == -1 && look(total).first == total);
    // wrong ones: the list ends there, and says so
    const int where = below(g_E + 1);
    const int32_t wrong[] = {-1, g_rows + 1, INT_MAX, INT_MIN};
    g_offsets[where] = wrong[below(4)];
    g_later = g_offsets;
    for (int i = 0; i < 3; ++i) {
      const int at = below(total + 2);
      g_error = 0;
      const RowTiles r = look(at);
      within(r, at);
      EXPECT(r.e < where && (r.e >= 0 || g_error == 1));
    }
    // ones that change, from what was there before to the right ones, at any of the loads
    for (int i = 0; i < 6; ++i) {
      g_offsets.assign(g_E + 1, 0);
      if (i & 1)
        for (auto &o : g_offsets) o = below(2) ? below(g_rows + 1) : (int32_t)g();
      if (i >= 2) g_offsets[0] = 0;
      g_later = right;
      g_left = below(64 * 6);
      const int at = below(total + 2);
      within(look(at), at);
    }
  }
  std::printf("failures %d\n", g_fail);
  return g_fail != 0;
}
