// Host-only driver of the key/value cache's C-ABI layer (csrc/api_kv4.cpp) for
// AddressSanitizer and UndefinedBehaviorSanitizer builds with the host compiler.  The device
// launchers are stubs that count their calls, so every entry point's validation and marshalling
// runs without a GPU.  Exit status 0 when every expectation holds.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/trellis_kv4.h"
#include "../../trellis_coded_bit_amd/csrc/abi.h"
#include "../../trellis_coded_bit_amd/csrc/launch.h"
#include "../../trellis_coded_bit_amd/csrc/launch_kv4.h"

static int g_launches = 0, g_fail = 0;
static char g_text[512];
#define EXPECT(c)                                                                                            \
  do {                                                                                                       \
    if (!(c)) {                                                                                              \
      std::fprintf(stderr, "expectation failed at line %d: %s (last error: %s)\n", __LINE__, #c, g_text);   \
      ++g_fail;                                                                                              \
    }                                                                                                        \
  } while (0)

namespace trellis {
int abi_fail(int status, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_text, sizeof(g_text), fmt, ap);
  va_end(ap);
  return status;
}
void abi_clear() { g_text[0] = 0; }
int abi_hip_status(hipError_t e, const char *what) {
  return e == hipSuccess ? TRELLIS_OK : abi_fail(TRELLIS_EHIP, "%s: %d", what, (int)e);
}
static hipError_t g_next = hipSuccess;
static hipError_t launched() { ++g_launches; return g_next; }
hipError_t launch_kv4_append(const trellis_kv4_cache &c, int, const trellis_kv4_batch &b, int, const Kv4Rows &k,
                             const Kv4Rows &v, uint32_t *e, hipStream_t) {
  EXPECT(c.pool && b.rows > 0 && k.p && v.p && e);
  return launched();
}
hipError_t launch_kv4_read(const trellis_kv4_cache &, int, const trellis_kv4_batch &b, int, void *k, void *v, uint32_t *e,
                           hipStream_t) {
  EXPECT(b.rows > 0 && k && v && e);
  return launched();
}
size_t kv4_attn_workspace_bytes(const trellis_kv4_cache &, const trellis_kv4_batch &b, int n) {
  return kWsReserved + (size_t)b.rows * n;
}
hipError_t launch_kv4_attn(const Kv4Attn &a, void *ws, hipStream_t) {
  EXPECT(a.q.p && a.y && ws && a.b.rows > 0);
  return launched();
}
size_t kv4_pages_workspace_bytes(int n_pages, int n) { return kWsReserved + (size_t)4 * n_pages + (size_t)4 * n; }
hipError_t launch_kv4_reserve(const Kv4Pages &p, void *, hipStream_t) { EXPECT(p.add); return launched(); }
hipError_t launch_kv4_fork(const Kv4Pages &p, void *, hipStream_t) { EXPECT(p.src && p.dst); return launched(); }
hipError_t launch_kv4_compact(const Kv4Pages &p, void *, hipStream_t) { EXPECT(p.src && p.dst && p.keep_cu); return launched(); }
hipError_t launch_kv4_free(const Kv4Pages &p, uint32_t *e, hipStream_t) { EXPECT(p.dst && e); return launched(); }
}  // namespace trellis

template <typename T>
static T *at(uintptr_t a) { return reinterpret_cast<T *>(a); }

int main() {
  const size_t big = (size_t)1 << 30;
  EXPECT(trellis_kv4_page_bytes(16, 8, 128) == 132u * 16 * 8);
  EXPECT(trellis_kv4_page_bytes(256, 1, 256) == 132u * 2 * 256);
  EXPECT(trellis_kv4_page_bytes(8, 8, 128) == 0 && trellis_kv4_page_bytes(48, 8, 128) == 0);
  EXPECT(trellis_kv4_page_bytes(16, 0, 128) == 0 && trellis_kv4_page_bytes(16, 1025, 128) == 0);
  EXPECT(trellis_kv4_page_bytes(16, 8, 64) == 0 && trellis_kv4_workspace_bytes() == trellis::kWsReserved);

  trellis_kv4_cache c{at<void>(0x10000), 2, 100, 16, 4, 128};
  trellis_kv4_batch b{at<int32_t>(0x20000), at<int32_t>(0x21000), nullptr, at<int32_t>(0x22000), 3, 10, 3, 3};
  void *k = at<void>(0x30000), *v = at<void>(0x40000), *ws = at<void>(0x100000);
  auto append = [&](const trellis_kv4_cache *cc, int layer, const trellis_kv4_batch *bb, int dt, const void *kk, int64_t row,
                    int64_t head, size_t nb, void *w) {
    return trellis_kv4_append(cc, layer, bb, dt, kk, row, head, v, 512, 128, w, nb, nullptr);
  };
  EXPECT(append(&c, 0, &b, 0, k, 512, 128, big, ws) == TRELLIS_OK && g_launches == 1);
  EXPECT(append(nullptr, 0, &b, 0, k, 512, 128, big, ws) == TRELLIS_EINVAL && g_text[0]);
  EXPECT(append(&c, 0, nullptr, 0, k, 512, 128, big, ws) == TRELLIS_EINVAL);
  EXPECT(append(&c, 2, &b, 0, k, 512, 128, big, ws) == TRELLIS_EINVAL);
  EXPECT(append(&c, -1, &b, 0, k, 512, 128, big, ws) == TRELLIS_EINVAL);
  EXPECT(append(&c, 0, &b, 2, k, 512, 128, big, ws) == TRELLIS_EINVAL);
  EXPECT(append(&c, 0, &b, 0, nullptr, 512, 128, big, ws) == TRELLIS_EINVAL);
  EXPECT(append(&c, 0, &b, 0, at<void>(0x30008), 512, 128, big, ws) == TRELLIS_EALIGN);
  EXPECT(append(&c, 0, &b, 0, k, 516, 128, big, ws) == TRELLIS_EALIGN);
  EXPECT(append(&c, 0, &b, 0, k, -512, 128, big, ws) == TRELLIS_EINVAL);
  EXPECT(append(&c, 0, &b, 0, k, 512, 128, 100, ws) == TRELLIS_EWORKSPACE);
  EXPECT(append(&c, 0, &b, 0, k, 512, 128, big, nullptr) == TRELLIS_EWORKSPACE);
  EXPECT(append(&c, 0, &b, 0, k, 512, 128, big, at<void>(0x100010)) == TRELLIS_EWORKSPACE);
  for (int f = 0; f < 8; ++f) {  // bad caches and batches
    trellis_kv4_cache d = c;
    trellis_kv4_batch e = b;
    int want = TRELLIS_EINVAL;
    switch (f) {
      case 0: d.page_size = 24; break;
      case 1: d.n_pages = 0; break;
      case 2: d.pool = at<void>(0x10010); want = TRELLIS_EALIGN; break;
      case 3: e.n_slots = 0; break;
      case 4: e.max_pages = 1 << 27; break;
      case 5: e.rows = -1; break;
      case 6: e.cu = nullptr; break;
      case 7: e.table = at<int32_t>(0x20002); want = TRELLIS_EALIGN; break;
    }
    EXPECT(append(&d, 0, &e, 0, k, 512, 128, big, ws) == want);
    EXPECT(trellis_kv4_read(&d, 0, &e, 0, k, v, ws, big, nullptr) == want);
    EXPECT(trellis_kv4_attn(&d, 0, &e, 0, k, 512, 128, 4, 1.f, 0, 0, 0, v, nullptr, ws, big, nullptr) == want);
    EXPECT(trellis_kv4_attn_workspace_bytes(&d, &e, 4) == 0);
  }
  trellis_kv4_batch none = b;
  none.rows = 0;
  EXPECT(append(&c, 0, &none, 0, nullptr, 0, 0, 0, nullptr) == TRELLIS_OK && g_launches == 1);
  none.rows = 2;
  none.n_seq = 0;
  EXPECT(append(&c, 0, &none, 0, k, 512, 128, big, ws) == TRELLIS_EINVAL);

  EXPECT(trellis_kv4_read(&c, 1, &b, 1, k, v, ws, big, nullptr) == TRELLIS_OK && g_launches == 2);
  EXPECT(trellis_kv4_read(&c, 1, &b, 1, k, nullptr, ws, big, nullptr) == TRELLIS_EINVAL);

  auto attn = [&](int heads, float scale, int window, int sinks, int most, void *y, size_t nb) {
    return trellis_kv4_attn(&c, 0, &b, 0, k, heads * 128, 128, heads, scale, window, sinks, most, y, nullptr, ws, nb, nullptr);
  };
  EXPECT(attn(8, 0.1f, 0, 0, 0, v, big) == TRELLIS_OK && g_launches == 3);
  EXPECT(attn(6, 0.1f, 0, 0, 0, v, big) == TRELLIS_EINVAL && attn(0, 0.1f, 0, 0, 0, v, big) == TRELLIS_EINVAL);
  EXPECT(attn(4 * 65, 0.1f, 0, 0, 0, v, big) == TRELLIS_EINVAL);
  EXPECT(attn(8, INFINITY, 0, 0, 0, v, big) == TRELLIS_EINVAL && attn(8, NAN, 0, 0, 0, v, big) == TRELLIS_EINVAL);
  EXPECT(attn(8, 0.1f, -1, 0, 0, v, big) == TRELLIS_EINVAL && attn(8, 0.1f, 0, -1, 0, v, big) == TRELLIS_EINVAL);
  EXPECT(attn(8, 0.1f, 0, 0, -1, v, big) == TRELLIS_EINVAL);
  EXPECT(attn(8, 0.1f, 0, 0, 0, k, big) == TRELLIS_EINVAL);                 // y is q
  EXPECT(attn(8, 0.1f, 0, 0, 0, at<void>(0x30010), big) == TRELLIS_EINVAL); // y inside q
  EXPECT(attn(8, 0.1f, 0, 0, 0, v, trellis_kv4_attn_workspace_bytes(&c, &b, 8) - 1) == TRELLIS_EWORKSPACE);

  int32_t *table = at<int32_t>(0x50000), *lens = at<int32_t>(0x51000), *ref = at<int32_t>(0x52000), *l = at<int32_t>(0x53000);
  const size_t need = trellis_kv4_pages_workspace_bytes(&c, 3);
  EXPECT(need > 0 && trellis_kv4_pages_workspace_bytes(nullptr, 3) == 0 && trellis_kv4_pages_workspace_bytes(&c, -1) == 0);
  EXPECT(trellis_kv4_reserve(&c, table, lens, 4, 10, ref, nullptr, l, 3, ws, need, nullptr) == TRELLIS_OK);
  EXPECT(trellis_kv4_reserve(&c, table, lens, 4, 10, ref, nullptr, nullptr, 3, ws, need, nullptr) == TRELLIS_EINVAL);
  EXPECT(trellis_kv4_reserve(&c, table, lens, 4, 10, ref, nullptr, l, 5, ws, big, nullptr) == TRELLIS_EINVAL);
  EXPECT(trellis_kv4_reserve(&c, table, lens, 4, 10, ref, at<int32_t>(0x53002), l, 3, ws, need, nullptr) == TRELLIS_EALIGN);
  EXPECT(trellis_kv4_fork(&c, table, lens, 4, 10, ref, l, l, 3, ws, need, nullptr) == TRELLIS_OK);
  EXPECT(trellis_kv4_fork(&c, table, lens, 4, 10, nullptr, l, l, 3, ws, need, nullptr) == TRELLIS_EINVAL);
  EXPECT(trellis_kv4_fork(&c, table, lens, 4, 10, ref, l, nullptr, 3, ws, need, nullptr) == TRELLIS_EINVAL);
  EXPECT(trellis_kv4_fork(&c, table, lens, 4, 10, ref, l, l, 3, ws, need - 1, nullptr) == TRELLIS_EWORKSPACE);
  EXPECT(trellis_kv4_fork(&c, table, lens, 1 << 19, 10, ref, l, l, 3, ws, need, nullptr) == TRELLIS_EINVAL);
  EXPECT(trellis_kv4_fork(&c, nullptr, nullptr, 4, 10, nullptr, nullptr, nullptr, 0, nullptr, 0, nullptr) == TRELLIS_EINVAL);
  EXPECT(trellis_kv4_fork(&c, table, lens, 4, 10, ref, nullptr, nullptr, 0, nullptr, 0, nullptr) == TRELLIS_OK);
  EXPECT(trellis_kv4_compact(&c, table, lens, 4, 10, ref, l, l, 2, l, l, 7, ws, need, nullptr) == TRELLIS_OK);
  EXPECT(trellis_kv4_compact(&c, table, lens, 4, 10, ref, l, l, 2, nullptr, l, 0, ws, need, nullptr) == TRELLIS_OK);
  EXPECT(trellis_kv4_compact(&c, table, lens, 4, 10, ref, l, l, 2, nullptr, l, 7, ws, need, nullptr) == TRELLIS_EINVAL);
  EXPECT(trellis_kv4_compact(&c, table, lens, 4, 10, ref, l, l, 2, l, l, -1, ws, need, nullptr) == TRELLIS_EINVAL);
  EXPECT(trellis_kv4_free(&c, table, lens, 4, 10, ref, l, 4, ws, big, nullptr) == TRELLIS_OK);
  EXPECT(trellis_kv4_free(&c, table, at<int32_t>(0x51001), 4, 10, ref, l, 4, ws, big, nullptr) == TRELLIS_EALIGN);
  EXPECT(trellis_kv4_free(&c, table, lens, 4, 10, ref, nullptr, 4, ws, big, nullptr) == TRELLIS_EINVAL);
  trellis::g_next = hipErrorInvalidValue;
  EXPECT(attn(8, 0.1f, 0, 0, 0, v, big) == TRELLIS_EHIP);
  std::printf("launches %d failures %d\n", g_launches, g_fail);
  return g_fail != 0;
}
