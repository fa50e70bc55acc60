// Attention over the 4-bit key/value cache.
#include "kv4_device.h"

namespace trellis {

namespace {

struct AttnArgs {
  Kv4Attn a;
  uint32_t *errword;
};

// One wave per (row, query head).  The rotated query stays in LDS; 64 keys at a time, a key a
// lane, with a running maximum and sum; then each lane gathers its share of the head's
// elements over the 64 values.
template <bool BF, int NB>
__global__ __launch_bounds__(256) void kv4_attn_simple_kernel(AttnArgs g) {
  const Kv4Attn &a = g.a;
  constexpr int D = 128 * NB;
  __shared__ float qs[4][D];
  __shared__ float ps[4][64];
  __shared__ const char *bases[4][64];
  __shared__ int places[4][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const long long task = (long long)blockIdx.x * 4 + wave;
  const bool live = task < (long long)a.b.rows * a.n_q_heads;
  const int row = live ? (int)(task / a.n_q_heads) : 0, head = live ? (int)(task % a.n_q_heads) : 0;
  const int kvh = head / (a.n_q_heads / a.c.n_kv_heads), T = a.c.page_size;
  int len = 0, pos = -1, slot = 0;
  const int s = kv4_seq_of(a.b.cu, a.b.n_seq, row, lane & 15);
  if (s < a.b.n_seq) {
    slot = a.b.slots ? a.b.slots[s] : s;
    if ((uint32_t)slot < (uint32_t)a.b.n_slots) {
      len = a.b.lens[slot];
      if (len < 0 || len > (long long)a.b.max_pages * T) {
        if (lane == 0) kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);
        len = 0;
      }
      pos = len - a.b.cu[s + 1] + row;
    } else if (lane == 0) {
      kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);
    }
  } else if (lane == 0) {
    kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);
  }
  const uint16_t *q = static_cast<const uint16_t *>(a.q.p) + row * a.q.row_stride + head * a.q.head_stride;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float x = kv4_widen<BF>(q[nb * 128 + lane]), y = kv4_widen<BF>(q[nb * 128 + 64 + lane]);
    wave_fwht128(x, y);
    qs[wave][nb * 128 + lane] = x * kRsqrt128 * a.scale;
    qs[wave][nb * 128 + 64 + lane] = y * kRsqrt128 * a.scale;
  }
  const Kv4Chunk ch{T, NB};
  const int end = live ? (pos + 1 < len ? pos + 1 : len) : 0;
  const int lo = a.window ? (pos - a.window + 1 > 0 ? pos - a.window + 1 : 0) : 0;
  float m = -__builtin_inff(), l = 0.f, o0[NB], o1[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) o0[nb] = o1[nb] = 0.f;
  for (int j0 = 0; j0 < end; j0 += 64) {
    if (j0 + 63 < lo && j0 >= a.sinks) {
      j0 = (lo / 64 - 1) * 64;
      continue;
    }
    const int j = j0 + lane;
    float sc = -__builtin_inff();
    const char *base = nullptr;
    if (j < end && (j >= lo || j < a.sinks)) {
      const int page = a.b.table[(size_t)slot * a.b.max_pages + j / T];
      if ((uint32_t)page < (uint32_t)a.c.n_pages) {
        base = kv4_chunk(a.c, a.layer, page, kvh);
        sc = 0.f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint32_t *w = reinterpret_cast<const uint32_t *>(base + ch.k_code(nb, j % T));
          float dot = 0.f;
          for (int t = 0; t < 16; ++t) {
            float v[8];
            kv4_values8(w[t], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = fmaf(v[e], qs[wave][nb * 128 + 8 * t + e], dot);
          }
          sc += dot * kv4_widen<true>(*reinterpret_cast<const uint16_t *>(base + ch.k_scale(nb, j % T)));
        }
      } else {
        kv4_error(g.errword, TRELLIS_KV4_ERR_BAD);
      }
    }
    float top = sc;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    const float m2 = fmaxf(m, top);
    const float mu = m2 == -__builtin_inff() ? 0.f : m2;
    const float f = __expf(m - mu), p = base ? __expf(sc - mu) : 0.f;
    float sum = p;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    l = l * f + sum;
    m = m2;
    ps[wave][lane] = p;
    bases[wave][lane] = base;
    places[wave][lane] = j % T;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      o0[nb] *= f;
      o1[nb] *= f;
    }
    for (int t = 0; t < 64; ++t) {
      const char *bt = bases[wave][t];
      if (!bt) continue;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const uint8_t w = *reinterpret_cast<const uint8_t *>(bt + ch.v_code(nb, places[wave][t]) + lane);
        const float pv = ps[wave][t] * kv4_widen<true>(*reinterpret_cast<const uint16_t *>(bt + ch.v_scale(nb, places[wave][t])));
        const floatx2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)w, 1.0f, 0);
        o0[nb] = fmaf(pv, v[0], o0[nb]);
        o1[nb] = fmaf(pv, v[1], o1[nb]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  if (!live) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t *y = static_cast<uint16_t *>(a.y) + ((size_t)row * a.n_q_heads + head) * D;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {  // the lane holds elements 2 lane, 2 lane + 1
    float x0 = o0[nb] * inv, x1 = o1[nb] * inv;
    wave_fwht128(x0, x1);
    const uint32_t w = (uint32_t)kv4_narrow<BF>(x0 * kRsqrt128) | ((uint32_t)kv4_narrow<BF>(x1 * kRsqrt128) << 16);
    *reinterpret_cast<uint32_t *>(y + nb * 128 + 2 * lane) = w;
  }
  if (a.lse && lane == 0) a.lse[(size_t)row * a.n_q_heads + head] = l == 0.f ? -__builtin_inff() : m + __logf(l);
}

}  // namespace

size_t kv4_attn_workspace_bytes(const trellis_kv4_cache &, const trellis_kv4_batch &, int) { return kWsReserved; }

hipError_t launch_kv4_attn(const Kv4Attn &a, void *ws, hipStream_t stream) {
  const AttnArgs g{a, static_cast<uint32_t *>(ws)};
  const unsigned grid = (unsigned)(((long long)a.b.rows * a.n_q_heads + 3) / 4);
  const bool bf = a.dtype == TRELLIS_KV4_BF16;
  if (a.c.head_dim == 128) {
    if (bf) kv4_attn_simple_kernel<true, 1><<<grid, 256, 0, stream>>>(g);
    else kv4_attn_simple_kernel<false, 1><<<grid, 256, 0, stream>>>(g);
  } else {
    if (bf) kv4_attn_simple_kernel<true, 2><<<grid, 256, 0, stream>>>(g);
    else kv4_attn_simple_kernel<false, 2><<<grid, 256, 0, stream>>>(g);
  }
  return hipGetLastError();
}

}  // namespace trellis
