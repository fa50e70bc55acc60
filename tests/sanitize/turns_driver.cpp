// Host-only driver of the C-ABI layer (csrc/api.cpp, api_kv4.cpp, api_f8.cpp) under several host
// threads: the calls that use a workspace's scratch are made by all of them with one workspace, and
// with one of their own.  The launchers are stubs that take a while between their first and their last
// launch and count who else is in one with the same workspace meanwhile.  Exit status 0 when that is
// nobody and every call was accepted.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <functional>
#include <thread>
#include <vector>

#include "../../include/trellis.h"
#include "../../include/trellis_f8.h"
#include "../../include/trellis_kv4.h"
#include "../../include/trellis_route.h"
#include "../../trellis_coded_bit_amd/csrc/launch.h"
#include "../../trellis_coded_bit_amd/csrc/launch_f8.h"
#include "../../trellis_coded_bit_amd/csrc/launch_kv4.h"

extern "C" const char *hipGetErrorString(hipError_t) { return "stub HIP error"; }

// Workspaces are addresses kFirst + i * kStep that nothing dereferences.
constexpr int kThreads = 4;
constexpr uintptr_t kFirst = 0x7000000000, kStep = 1 << 20;
static std::atomic<int> g_inside[kThreads + 1], g_together{0}, g_launches{0}, g_refused{0};

static hipError_t launches(const void *ws) {
  std::atomic<int> &in = g_inside[(reinterpret_cast<uintptr_t>(ws) - kFirst) / kStep];
  if (in.fetch_add(1)) ++g_together;
  std::this_thread::sleep_for(std::chrono::microseconds(30));
  if (in.fetch_sub(1) != 1) ++g_together;
  ++g_launches;
  return hipSuccess;
}

namespace trellis {
hipError_t launch_decode_tiles(const int16_t *, int, int, int, uint16_t *, uint16_t *, hipStream_t) { return hipSuccess; }
hipError_t launch_decode_tiles_e4m3(const int16_t *, int, int, int, uint8_t *, hipStream_t) { return hipSuccess; }
hipError_t launch_had128(const void *, int, int, int, const uint16_t *, const float *, int, float, void *, int, hipStream_t) { return hipSuccess; }
size_t gemv_workspace_bytes(const GemvLaunch &) { return kWsReserved; }
size_t gemv_workspace_bytes(int, int, int, int) { return kWsReserved; }
hipError_t launch_gemv(const GemvLaunch &, void *ws, size_t, hipStream_t) { return launches(ws); }
hipError_t noalloc_scratch(void **) { return hipErrorNotInitialized; }
size_t moe_mlp_workspace_bytes(int, int, int, int) { return kWsReserved; }
hipError_t launch_moe_mlp(const MlpLaunch &, void *ws, size_t, hipStream_t) { return launches(ws); }
size_t encode_workspace_bytes(int) { return kWsReserved; }
hipError_t launch_encode_tiles(const float *, int, int, int, int16_t *, uint16_t *, void *ws, size_t, hipStream_t) { return launches(ws); }
size_t gemm_workspace_bytes(int, int, int) { return kWsReserved; }
hipError_t launch_gemm(const trellis_linear &, const uint16_t *, int, uint16_t *, void *ws, size_t, hipStream_t) { return launches(ws); }
size_t gemm_fp8_workspace_bytes(int, int, int) { return kWsReserved; }
hipError_t launch_gemm_fp8(const trellis_linear &, const uint16_t *, int, uint16_t *, void *ws, size_t, hipStream_t) { return launches(ws); }
int micro_cus() { return 256; }
hipError_t launch_micro_stream_read(const void *, size_t, int, uint32_t *, hipStream_t) { return hipSuccess; }
hipError_t launch_micro_valu(int, int, int, uint64_t *, uint64_t *, uint32_t *, hipStream_t, int *) { return hipSuccess; }
hipError_t launch_micro_mfma(int, int, int, uint64_t *, uint64_t *, float *, hipStream_t, int *) { return hipSuccess; }

hipError_t launch_kv4_append(const trellis_kv4_cache &, int, const trellis_kv4_batch &, int, const Kv4Rows &, const Kv4Rows &, uint32_t *,
                             hipStream_t) { return hipSuccess; }
hipError_t launch_kv4_read(const trellis_kv4_cache &, int, const trellis_kv4_batch &, int, void *, void *, uint32_t *, hipStream_t) { return hipSuccess; }
size_t kv4_attn_workspace_bytes(const trellis_kv4_cache &, const trellis_kv4_batch &, int) { return kWsReserved; }
hipError_t launch_kv4_attn(const Kv4Attn &, void *ws, hipStream_t) { return launches(ws); }
size_t kv4_pages_workspace_bytes(int, int) { return kWsReserved; }
hipError_t launch_kv4_reserve(const Kv4Pages &, void *ws, hipStream_t) { return launches(ws); }
hipError_t launch_kv4_fork(const Kv4Pages &, void *ws, hipStream_t) { return launches(ws); }
hipError_t launch_kv4_compact(const Kv4Pages &, void *ws, hipStream_t) { return launches(ws); }
hipError_t launch_kv4_free(const Kv4Pages &, uint32_t *, hipStream_t) { return hipSuccess; }

hipError_t launch_f8_norm(const F8Norm &, hipStream_t) { return hipSuccess; }
hipError_t launch_f8_silu_mul(const F8Act &, hipStream_t) { return hipSuccess; }
size_t f8_gemm_workspace_bytes(const trellis_f8_linear &, int, bool) { return kWsReserved; }
hipError_t launch_f8_gemm(const F8Gemm &, void *ws, hipStream_t) { return launches(ws); }
size_t moe_sort_workspace_bytes(int, int, int) { return kWsReserved; }
hipError_t launch_moe_sort(const int32_t *, int, int, int, int32_t *, int32_t *, int32_t *, void *ws, hipStream_t) { return launches(ws); }
hipError_t launch_moe_gather(const void *, int64_t, int, int64_t, const int32_t *, int, int, void *, uint32_t *, hipStream_t) { return hipSuccess; }
hipError_t launch_moe_combine(const MoeCombine &, uint32_t *, hipStream_t) { return hipSuccess; }
hipError_t launch_moe_combine_grad(const MoeCombine &, uint32_t *, hipStream_t) { return hipSuccess; }
}  // namespace trellis

template <typename T>
static T *at(uintptr_t a) { return reinterpret_cast<T *>(a); }

int main() {
  const size_t nb = trellis::kWsReserved;
  const trellis_linear L{at<int16_t>(0x100000), at<uint16_t>(0x200000), at<uint16_t>(0x300000), nullptr, nullptr, 2, 128, 128, 2};
  const trellis_gemv_item item{L, at<uint16_t>(0x400000), at<uint16_t>(0x500000)};
  const trellis_kv4_cache c{at<void>(0x10000), 2, 100, 16, 4, 128};
  const trellis_kv4_batch b{at<int32_t>(0x20000), at<int32_t>(0x21000), nullptr, at<int32_t>(0x22000), 3, 10, 3, 3};
  const trellis_f8_linear F{at<uint8_t>(0x100000000), at<float>(0x200000000), 1, 256, 256};
  trellis_f8_linear E = F;
  E.n_experts = 4;
  uint16_t *x = at<uint16_t>(0x1000000), *y = at<uint16_t>(0x6000000);
  int32_t *i0 = at<int32_t>(0x8000000), *i1 = at<int32_t>(0x9000000), *i2 = at<int32_t>(0xA000000), *i3 = at<int32_t>(0xB000000);
  uint8_t *q = at<uint8_t>(0x5000000);
  float *s = at<float>(0x5800000);
  const std::vector<std::function<int(void *)>> calls = {
      [&](void *ws) { return trellis_gemv(&L, x, 1, y, ws, nb, nullptr); },
      [&](void *ws) { return trellis_gemv_list(&item, 1, 2, ws, nb, nullptr); },
      [&](void *ws) { return trellis_gemm(&L, x, 64, y, ws, nb, nullptr); },
      [&](void *ws) { return trellis_gemm_fp8(&L, x, 64, y, ws, nb, nullptr); },
      [&](void *ws) { return trellis_moe_gemv(&L, 1, i0, 2, 128, 128, x, 0, nullptr, nullptr, -1, y, ws, nb, nullptr); },
      [&](void *ws) { return trellis_moe_mlp(&L, &L, 1, 1, i0, s, 2, 128, 128, x, x, nullptr, x, nullptr, nullptr, y, ws, nb, nullptr); },
      [&](void *ws) { return trellis_encode_tiles(s, 3, 2, 1, at<int16_t>(0x6000000), nullptr, ws, nb, nullptr); },
      [&](void *ws) { return trellis_kv4_attn(&c, 0, &b, 0, x, 512, 128, 4, 1.f, 0, 0, 0, y, nullptr, ws, nb, nullptr); },
      [&](void *ws) { return trellis_kv4_reserve(&c, i0, i1, 3, 10, i2, nullptr, i3, 3, ws, nb, nullptr); },
      [&](void *ws) { return trellis_kv4_fork(&c, i0, i1, 3, 10, i2, i3, i3, 1, ws, nb, nullptr); },
      [&](void *ws) { return trellis_kv4_compact(&c, i0, i1, 3, 10, i2, i3, i3, 1, i3, i3, 5, ws, nb, nullptr); },
      [&](void *ws) { return trellis_f8_gemm(&F, q, 256, s, 2, 5, 0, y, 256, ws, nb, nullptr); },
      [&](void *ws) { return trellis_f8_moe_gemm(&E, q, 256, s, 2, 5, i0, nullptr, 1, 5, 0, y, 256, ws, nb, nullptr); },
      [&](void *ws) { return trellis_moe_sort(i0, 7, 3, 8, i1, i2, i3, ws, nb, nullptr); },
  };
  const int n = (int)calls.size(), rounds = 20;
  std::vector<std::thread> threads;
  for (int t = 0; t < kThreads; ++t)
    threads.emplace_back([&, t] {
      for (int r = 0; r < rounds; ++r)
        for (int i = 0; i < n; ++i) {
          // every other call with the shared workspace, the threads at different calls
          const uintptr_t own = (i + r) & 1 ? (uintptr_t)(t + 1) : 0;
          const int st = calls[(i * (t + 1) + 3 * t + r) % n](at<void>(kFirst + own * kStep));
          if (st) {
            std::fprintf(stderr, "call %d refused: %d (%s)\n", (i * (t + 1) + 3 * t + r) % n, st, trellis_last_error());
            ++g_refused;
          }
        }
    });
  for (std::thread &t : threads) t.join();
  // each call once more on its own: the threads' strides need not have reached all of them
  for (const auto &call : calls) g_refused += call(at<void>(kFirst)) != 0;
  std::printf("launches %d of %d, refused %d, together %d\n", g_launches.load(), kThreads * rounds * n + n, g_refused.load(), g_together.load());
  return g_together || g_refused || g_launches != kThreads * rounds * n + n;
}
