// Host-only driver of the C-ABI layer of the block-scaled FP8 operators and the routed tokens
// (csrc/api_f8.cpp) for AddressSanitizer and UndefinedBehaviorSanitizer builds with the host
// compiler.  The device launchers are stubs that count their calls, so every entry point's
// validation and marshalling runs without a GPU.  Exit status 0 when every expectation holds.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/trellis_f8.h"
#include "../../include/trellis_route.h"
#include "../../trellis_coded_bit_amd/csrc/abi.h"
#include "../../trellis_coded_bit_amd/csrc/launch.h"
#include "../../trellis_coded_bit_amd/csrc/launch_f8.h"

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
static F8Gemm g_gemm;
hipError_t launch_f8_norm(const F8Norm &a, hipStream_t) {
  EXPECT(a.x && (a.out.q || a.out.y) && a.rows > 0 && a.x_row >= a.n);
  return launched();
}
hipError_t launch_f8_silu_mul(const F8Act &a, hipStream_t) {
  EXPECT(a.x && (a.out.q || a.out.y) && a.rows > 0 && a.x_row >= 2 * a.n);
  return launched();
}
size_t f8_gemm_workspace_bytes(const trellis_f8_linear &, int rows, bool) { return kWsReserved + (size_t)rows * 4; }
hipError_t launch_f8_gemm(const F8Gemm &a, void *ws, hipStream_t) {
  EXPECT(a.q && a.s && a.y && ws && a.rows > 0 && a.n_q > 0);
  g_gemm = a;
  return launched();
}
size_t moe_sort_workspace_bytes(int tokens, int top, int) { return kWsReserved + (size_t)tokens * top; }
hipError_t launch_moe_sort(const int32_t *, int, int, int, int32_t *offsets, int32_t *, int32_t *, void *ws, hipStream_t) {
  EXPECT(offsets && ws);
  return launched();
}
hipError_t launch_moe_gather(const void *, int64_t, int, int64_t, const int32_t *order, int rows, int, void *out, uint32_t *e, hipStream_t) {
  EXPECT(order && out && e && rows > 0);
  return launched();
}
hipError_t launch_moe_combine(const MoeCombine &a, uint32_t *e, hipStream_t) {
  EXPECT(a.out && a.inverse && e && a.tokens > 0);
  return launched();
}
hipError_t launch_moe_combine_grad(const MoeCombine &a, uint32_t *e, hipStream_t) {
  EXPECT(a.d_out && a.inverse && e && a.tokens > 0 && (!a.d_weights || a.y));
  return launched();
}
}  // namespace trellis

template <typename T>
static T *at(uintptr_t a) { return reinterpret_cast<T *>(a); }

int main() {
  const size_t big = (size_t)1 << 40;
  void *ws = at<void>(0x7000000000);
  void *x = at<void>(0x1000000), *r = at<void>(0x2000000), *g = at<void>(0x3000000), *h = at<void>(0x4000000),
       *y = at<void>(0x6000000);
  uint8_t *q = at<uint8_t>(0x5000000);
  float *s = at<float>(0x5800000);

  auto norm = [&](int dt, const void *xx, int64_t row, const void *res, int rows, int n, float eps, void *hh, uint8_t *qq, float *ss,
                  void *yy) { return trellis_f8_norm(dt, xx, row, res, g, rows, n, eps, hh, qq, ss, yy, nullptr); };
  EXPECT(norm(0, x, 256, r, 4, 256, 1e-6f, h, q, s, y) == TRELLIS_OK && g_launches == 1);
  EXPECT(norm(1, x, 264, nullptr, 4, 256, 1e-6f, nullptr, nullptr, nullptr, y) == TRELLIS_OK);
  EXPECT(norm(0, x, 256, r, 4, 256, 1e-6f, r, q, s, nullptr) == TRELLIS_OK);                    // the residual in place
  EXPECT(norm(0, x, 256, r, 4, 256, 1e-6f, x, q, s, nullptr) == TRELLIS_OK && g_launches == 4); // x in place
  EXPECT(norm(0, x, 264, r, 4, 256, 1e-6f, x, q, s, nullptr) == TRELLIS_EINVAL);                // x strided
  EXPECT(norm(0, x, 7, r, 1, 256, 1e-6f, x, q, s, nullptr) == TRELLIS_OK);                      // one row: no stride
  EXPECT(norm(2, x, 256, r, 4, 256, 1e-6f, h, q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, nullptr, 256, r, 4, 256, 1e-6f, h, q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, at<void>(0x1000008), 256, r, 4, 256, 1e-6f, h, q, s, y) == TRELLIS_EALIGN);
  EXPECT(norm(0, x, 260, r, 4, 256, 1e-6f, h, q, s, y) == TRELLIS_EALIGN);
  EXPECT(norm(0, x, 248, r, 4, 256, 1e-6f, h, q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, -256, r, 4, 256, 1e-6f, h, q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, 256, r, -1, 256, 1e-6f, h, q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, at<void>(big), 32768, nullptr, (1 << 22) - 1, 32768, 1e-6f, nullptr, nullptr, nullptr, at<void>(4 * big)) == TRELLIS_OK && --g_launches == 5);
  EXPECT(norm(0, at<void>(big), 32768, nullptr, 1 << 22, 32768, 1e-6f, nullptr, nullptr, nullptr, at<void>(4 * big)) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, 256, r, 4, 250, 1e-6f, h, q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, 40000, r, 4, 32784, 1e-6f, h, q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, 256, r, 4, 256, 0.f, h, q, s, y) == TRELLIS_EINVAL && norm(0, x, 256, r, 4, 256, NAN, h, q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, 256, r, 4, 256, INFINITY, h, q, s, y) == TRELLIS_EINVAL && norm(0, x, 256, r, 4, 256, 1e-39f, h, q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, 256, r, 4, 256, 1e-6f, h, nullptr, nullptr, nullptr) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, 256, r, 4, 256, 1e-6f, h, q, nullptr, y) == TRELLIS_EINVAL && norm(0, x, 256, r, 4, 256, 1e-6f, h, nullptr, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, 256, r, 4, 256, 1e-6f, h, q, s, h) == TRELLIS_EINVAL && norm(0, x, 256, r, 4, 256, 1e-6f, h, q, s, x) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, 256, r, 4, 256, 1e-6f, at<void>(0x2000010), q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, x, 256, r, 4, 256, 1e-6f, g, q, s, y) == TRELLIS_EINVAL);
  EXPECT(norm(0, nullptr, 0, nullptr, 0, 256, 1e-6f, nullptr, nullptr, nullptr, nullptr) == TRELLIS_OK && g_launches == 5);

  auto act = [&](int dt, const void *xx, int64_t row, int rows, int n, uint8_t *qq, float *ss, void *yy) {
    return trellis_f8_silu_mul(dt, xx, row, rows, n, qq, ss, yy, nullptr);
  };
  EXPECT(act(1, x, 512, 4, 256, q, s, y) == TRELLIS_OK && g_launches == 6);
  EXPECT(act(1, x, 511, 4, 256, q, s, y) == TRELLIS_EINVAL && act(1, x, 516, 4, 256, q, s, y) == TRELLIS_EALIGN);
  EXPECT(act(1, x, 512, 4, 24, q, s, y) == TRELLIS_EINVAL && act(1, x, 512, -1, 256, q, s, y) == TRELLIS_EINVAL);
  EXPECT(act(1, x, 512, 4, 256, nullptr, nullptr, nullptr) == TRELLIS_EINVAL && act(1, x, 512, 4, 256, q, s, x) == TRELLIS_EINVAL);
  EXPECT(act(1, x, 1 << 20, 1 << 30, 1 << 19, q, s, y) == TRELLIS_EINVAL);

  trellis_f8_linear L{at<uint8_t>(0x100000000), at<float>(0x200000000), 1, 272, 300};
  const size_t need = trellis_f8_gemm_workspace_bytes(&L, 5);
  EXPECT(need == trellis::kWsReserved + 20 && trellis_f8_gemm_workspace_bytes(nullptr, 5) == 0 && trellis_f8_gemm_workspace_bytes(&L, -1) == 0);
  auto gemm = [&](const trellis_f8_linear *l, const uint8_t *qq, int64_t qr, const float *ss, int64_t sr, int M, int dt, void *yy, int64_t yr,
                  size_t nb, void *w) { return trellis_f8_gemm(l, qq, qr, ss, sr, M, dt, yy, yr, w, nb, nullptr); };
  g_launches = 0;
  EXPECT(gemm(&L, q, 272, s, 3, 5, 0, y, 300, need, ws) == TRELLIS_OK && g_launches == 1);
  EXPECT(gemm(&L, q, 288, s, 7, 5, 1, y, 301, need, ws) == TRELLIS_OK);
  EXPECT(gemm(&L, q, -5, s, -5, 1, 1, y, -5, need, ws) == TRELLIS_OK && trellis::g_gemm.q_row == 0 && trellis::g_gemm.y_row == 0);
  EXPECT(gemm(&L, nullptr, 0, nullptr, 0, 0, 1, nullptr, 0, 0, nullptr) == TRELLIS_OK && g_launches == 3);
  EXPECT(gemm(&L, q, 256, s, 3, 5, 0, y, 300, need, ws) == TRELLIS_EINVAL && gemm(&L, q, 280, s, 3, 5, 0, y, 300, need, ws) == TRELLIS_EALIGN);
  EXPECT(gemm(&L, q, 272, s, 2, 5, 0, y, 300, need, ws) == TRELLIS_EINVAL && gemm(&L, q, 272, s, 3, 5, 0, y, 299, need, ws) == TRELLIS_EINVAL);
  EXPECT(gemm(&L, q, 272, s, 3, 5, 2, y, 300, need, ws) == TRELLIS_EINVAL && gemm(&L, q, 272, s, 3, -1, 0, y, 300, need, ws) == TRELLIS_EINVAL);
  EXPECT(gemm(&L, at<uint8_t>(0x5000008), 272, s, 3, 5, 0, y, 300, need, ws) == TRELLIS_EALIGN);
  EXPECT(gemm(&L, q, 272, s, 3, 5, 0, q, 300, need, ws) == TRELLIS_EINVAL && gemm(&L, q, 272, s, 3, 5, 0, (void *)L.w, 300, need, ws) == TRELLIS_EINVAL);
  EXPECT(gemm(&L, q, 272, s, 3, 5, 0, y, 300, need - 1, ws) == TRELLIS_EWORKSPACE && gemm(&L, q, 272, s, 3, 5, 0, y, 300, need, nullptr) == TRELLIS_EWORKSPACE);
  for (int f = 0; f < 7; ++f) {
    trellis_f8_linear d = L;
    int want = TRELLIS_EINVAL;
    switch (f) {
      case 0: d.in_features = 264; break;
      case 1: d.in_features = 0; break;
      case 2: d.out_features = 0; break;
      case 3: d.n_experts = 2; break;
      case 4: d.w = nullptr; break;
      case 5: d.w = at<uint8_t>(0x100000008); want = TRELLIS_EALIGN; break;
      case 6: d.scale = nullptr; break;
    }
    EXPECT(gemm(&d, q, 272, s, 3, 5, 0, y, 300, big, ws) == want);
  }
  EXPECT(gemm(nullptr, q, 272, s, 3, 5, 0, y, 300, big, ws) == TRELLIS_EINVAL);
  {
    trellis_f8_linear d = L;
    d.out_features = 1 << 20;
    d.in_features = 1 << 20;
    EXPECT(gemm(&d, q, 1 << 20, s, 8192, 1 << 26, 0, y, 1 << 20, big, ws) == TRELLIS_EINVAL);
  }

  trellis_f8_linear E = L;
  E.n_experts = 8;
  int32_t *off = at<int32_t>(0x8000000), *order = at<int32_t>(0x9000000), *inv = at<int32_t>(0xA000000), *ids = at<int32_t>(0xB000000);
  auto moe = [&](int n_q, const int32_t *o, const int32_t *ord, int per, int rows, size_t nb) {
    return trellis_f8_moe_gemm(&E, q, 272, s, 3, n_q, o, ord, per, rows, 0, y, 300, ws, nb, nullptr);
  };
  g_launches = 0;
  EXPECT(moe(4, off, order, 2, 8, big) == TRELLIS_OK && moe(8, off, nullptr, 1, 8, big) == TRELLIS_OK && g_launches == 2);
  EXPECT(moe(0, off, order, 2, 0, big) == TRELLIS_OK && g_launches == 2);
  EXPECT(moe(4, off, nullptr, 1, 8, big) == TRELLIS_EINVAL && moe(4, nullptr, order, 2, 8, big) == TRELLIS_EINVAL);
  EXPECT(moe(4, off, order, 0, 8, big) == TRELLIS_EINVAL && moe(0, off, order, 1, 8, big) == TRELLIS_EINVAL && moe(4, off, order, 2, -1, big) == TRELLIS_EINVAL);
  EXPECT(moe(4, at<int32_t>(0x8000002), order, 2, 8, big) == TRELLIS_EALIGN && moe(4, off, at<int32_t>(0x9000002), 2, 8, big) == TRELLIS_EALIGN);
  EXPECT(moe(4, off, order, 2, 8, trellis_f8_moe_gemm_workspace_bytes(&E, 8) - 1) == TRELLIS_EWORKSPACE);

  auto sort = [&](const int32_t *i, int tokens, int top, int e, int32_t *o, int32_t *ord, int32_t *in, size_t nb) {
    return trellis_moe_sort(i, tokens, top, e, o, ord, in, ws, nb, nullptr);
  };
  g_launches = 0;
  EXPECT(sort(ids, 7, 3, 8, off, order, inv, big) == TRELLIS_OK && g_launches == 1);
  EXPECT(sort(nullptr, 0, 3, 8, off, nullptr, nullptr, big) == TRELLIS_OK && g_launches == 2);  // offsets are zeros
  EXPECT(sort(ids, 7, 0, 8, off, order, inv, big) == TRELLIS_EINVAL && sort(ids, -1, 3, 8, off, order, inv, big) == TRELLIS_EINVAL);
  EXPECT(sort(ids, 7, 1025, 8, off, order, inv, big) == TRELLIS_EINVAL && sort(ids, 1 << 24, 2, 8, off, order, inv, big) == TRELLIS_EINVAL);
  EXPECT(sort(ids, 7, 3, 0, off, order, inv, big) == TRELLIS_EINVAL && sort(ids, 7, 3, 2049, off, order, inv, big) == TRELLIS_EINVAL);
  EXPECT(sort(nullptr, 7, 3, 8, off, order, inv, big) == TRELLIS_EINVAL && sort(ids, 7, 3, 8, nullptr, order, inv, big) == TRELLIS_EINVAL);
  EXPECT(sort(ids, 7, 3, 8, off, ids, inv, big) == TRELLIS_EINVAL && sort(ids, 7, 3, 8, off, order, order, big) == TRELLIS_EINVAL);
  EXPECT(sort(ids, 7, 3, 8, off, order, inv, trellis_moe_sort_workspace_bytes(7, 3, 8) - 1) == TRELLIS_EWORKSPACE);
  EXPECT(trellis_moe_sort_workspace_bytes(7, 0, 8) == 0 && trellis_moe_sort_workspace_bytes(7, 3, 0) == 0);

  auto gather = [&](const void *xx, int64_t row, int tokens, int64_t nb, const int32_t *ord, int rows, int per, void *o) {
    return trellis_moe_gather(xx, row, tokens, nb, ord, rows, per, o, ws, big, nullptr);
  };
  g_launches = 0;
  EXPECT(gather(x, 512, 4, 512, order, 8, 2, y) == TRELLIS_OK && gather(x, 516, 4, 12, order, 8, 2, y) == TRELLIS_OK && g_launches == 2);
  EXPECT(gather(x, 512, 4, 510, order, 8, 2, y) == TRELLIS_EINVAL && gather(x, 500, 4, 512, order, 8, 2, y) == TRELLIS_EINVAL);
  EXPECT(gather(x, 514, 4, 512, order, 8, 2, y) == TRELLIS_EALIGN && gather(x, 512, 4, 512, order, 8, 0, y) == TRELLIS_EINVAL);
  EXPECT(gather(x, 512, 4, 512, nullptr, 8, 2, y) == TRELLIS_EINVAL && gather(x, 512, 4, 512, order, 8, 2, x) == TRELLIS_EINVAL);
  EXPECT(gather(x, 512, 4, 512, nullptr, 0, 2, nullptr) == TRELLIS_OK && g_launches == 2);

  float *w = at<float>(0xC000000), *dw = at<float>(0xD000000);
  auto comb = [&](int dt, const void *yy, int rows, int n, const int32_t *in, int tokens, int top, const void *add, void *o) {
    return trellis_moe_combine(dt, yy, rows, n, in, w, tokens, top, add, o, ws, big, nullptr);
  };
  g_launches = 0;
  EXPECT(comb(0, y, 8, 264, inv, 4, 2, nullptr, x) == TRELLIS_OK && comb(1, y, 8, 264, inv, 4, 2, x, x) == TRELLIS_OK && g_launches == 2);
  EXPECT(comb(0, y, 8, 260, inv, 4, 2, nullptr, x) == TRELLIS_EINVAL && comb(0, y, 8, 264, nullptr, 4, 2, nullptr, x) == TRELLIS_EINVAL);
  EXPECT(comb(0, y, 8, 264, inv, 4, 2, nullptr, y) == TRELLIS_EINVAL && comb(0, y, 8, 264, inv, 4, 2, at<void>(0x1000010), x) == TRELLIS_EINVAL);
  EXPECT(comb(0, y, -1, 264, inv, 4, 2, nullptr, x) == TRELLIS_EINVAL && comb(3, y, 8, 264, inv, 4, 2, nullptr, x) == TRELLIS_EINVAL);
  EXPECT(comb(0, nullptr, 0, 264, inv, 4, 2, nullptr, x) == TRELLIS_OK && comb(0, nullptr, 0, 264, nullptr, 0, 2, nullptr, nullptr) == TRELLIS_OK && g_launches == 3);
  auto grad = [&](const void *d, const void *yy, void *dy, float *dww) {
    return trellis_moe_combine_grad(0, d, yy, 8, 264, inv, w, 4, 2, dy, dww, ws, big, nullptr);
  };
  g_launches = 0;
  EXPECT(grad(x, y, h, dw) == TRELLIS_OK && grad(x, y, y, dw) == TRELLIS_OK && grad(x, nullptr, h, nullptr) == TRELLIS_OK && g_launches == 3);
  EXPECT(grad(x, nullptr, h, dw) == TRELLIS_EINVAL && grad(nullptr, y, h, dw) == TRELLIS_EINVAL && grad(x, y, nullptr, dw) == TRELLIS_EINVAL);
  EXPECT(grad(x, y, x, dw) == TRELLIS_EINVAL && grad(x, y, h, w) == TRELLIS_EINVAL && grad(x, y, at<void>(0x6000010), dw) == TRELLIS_EINVAL);
  EXPECT(trellis_moe_combine_grad(0, x, y, 8, 264, inv, w, 4, 2, h, dw, ws, 8, nullptr) == TRELLIS_EWORKSPACE);
  trellis::g_next = hipErrorInvalidValue;
  EXPECT(comb(0, y, 8, 264, inv, 4, 2, nullptr, x) == TRELLIS_EHIP && act(1, x, 512, 4, 256, q, s, y) == TRELLIS_EHIP);
  std::printf("launches %d failures %d\n", g_launches, g_fail);
  return g_fail != 0;
}
