// The 4-bit key/value cache: append, read back, and the page operations.
#include "kv4_device.h"

namespace trellis {

namespace {

// ---------------------------------------------------------------------------------------
// Append and read
// ---------------------------------------------------------------------------------------
//
// Sixteen lanes hold one 128-block, eight elements a lane: one 16-byte load or store of 16-bit
// values, one word of codes.  A workgroup takes 16 consecutive rows and N of the (keys or values,
// head, block) kinds, so the 64-byte code rows of a kind fall next to each other in a page, and a
// row's page is looked up once for N blocks.  HBM bounds long calls (16-bit values in, a quarter of
// it out), with the rotation's vector instructions partly beside it (a copy without them takes 26.0 of
// 29.9 us); a few rows are bound by the chain of loads cu -> slot, length -> table before the store,
// which the rows' own loads overlap.  N = 4 where that still fills the card, else 1 (10338 rows of 8
// heads, append and read, 107 MB: 30.1 us at N = 4, 3.5 TB/s, 29.8 at N = 2, 33.7 at N = 1; N = 8 cost a
// ninth more).

template <bool BF, int N>
__global__ __launch_bounds__(256) void kv4_append_kernel(trellis_kv4_cache c, int layer, trellis_kv4_batch b, Kv4Rows k,
                                                         Kv4Rows v, uint32_t *errword) {
  const int NB = c.head_dim >> 7, kinds = 2 * c.n_kv_heads * NB;
  const int row = blockIdx.x * 16 + (threadIdx.x >> 4);
  if (row >= b.rows) return;  // (whole 16-lane groups leave together)
  const int i = threadIdx.x & 15, place = kv4_fwht16_place(i);
  const float sign = kv4_fwht16_sign(i) * kRsqrt128;
  u32x4 raw[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const Kv4Kind kind = kv4_kind(c, blockIdx.y * N + n);
    const Kv4Rows src = kind.is_v ? v : k;
    if (blockIdx.y * N + n < kinds)
      raw[n] = ldg(reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(src.p) + row * src.row_stride +
                                                   kind.head * src.head_stride + kind.nb * 128 + 8 * i));
  }
  const Kv4Place at = kv4_place(c, b, row, i);
  if (at.page < 0) {
    if (i == 0 && blockIdx.y == 0) kv4_error(errword, TRELLIS_KV4_ERR_BAD);
    return;
  }
  const Kv4Chunk ch{c.page_size, NB};
  const uint32_t chunk = ch.bytes();  // (a page's bytes fit 32 bits: 1024 heads of 132 * 2 * 256)
  char *page = kv4_chunk(c, layer, at.page < 0 ? 0 : at.page, 0);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (blockIdx.y * N + n >= kinds) break;
    const auto [head, nb, is_v] = kv4_kind(c, blockIdx.y * N + n);
    float x[8];
    kv4_unpack8<BF>(raw[n], x);
    kv4_fwht16_signed(x, i);
    // the largest magnitude as an integer: infinity is above every number, a NaN above infinity
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t m = __builtin_bit_cast(uint32_t, x[t]) & 0x7FFFFFFFu;
      top = m > top ? m : top;
    }
    top = kv4_max16(top);
    // the scale is rounded to bf16 first and the codes are taken against the rounded one
    uint16_t s = kv4_narrow<true>(__builtin_bit_cast(float, top) * kRsqrt128 * (1.f / 6.f));
    const float sf = kv4_widen<true>(s);
    uint32_t w = 0;
    if (top >= 0x7F800000u) {
      s = 0x7FC0;
    } else if (sf < 1.17549435e-38f) {
      s = 0;
    } else {
      const float inv = 1.f / sf * sign;
#pragma unroll
      for (int t = 0; t < 8; ++t) x[t] *= inv;
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], 1.0f, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], 1.0f, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], 1.0f, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], 1.0f, 3);
    }
    char *base = page + (uint32_t)head * chunk;
    *reinterpret_cast<uint32_t *>(base + (is_v ? ch.v_code(nb, at.at) : ch.k_code(nb, at.at)) + 4 * place) = w;
    if (i == 0) *reinterpret_cast<uint16_t *>(base + (is_v ? ch.v_scale(nb, at.at) : ch.k_scale(nb, at.at))) = s;
  }
}

template <bool BF, int N>
__global__ __launch_bounds__(256) void kv4_read_kernel(trellis_kv4_cache c, int layer, trellis_kv4_batch b, uint16_t *k,
                                                       uint16_t *v, uint32_t *errword) {
  const int NB = c.head_dim >> 7, kinds = 2 * c.n_kv_heads * NB;
  const int row = blockIdx.x * 16 + (threadIdx.x >> 4);
  if (row >= b.rows) return;
  const int i = threadIdx.x & 15, place = kv4_fwht16_place(i);
  const float sign = kv4_fwht16_sign(i) * kRsqrt128;
  const Kv4Place at = kv4_place(c, b, row, i);
  if (at.page < 0 && i == 0 && blockIdx.y == 0) kv4_error(errword, TRELLIS_KV4_ERR_BAD);
  const Kv4Chunk ch{c.page_size, NB};
  const uint32_t chunk = ch.bytes();  // (a page's bytes fit 32 bits: 1024 heads of 132 * 2 * 256)
  char *page = kv4_chunk(c, layer, at.page < 0 ? 0 : at.page, 0);
  uint32_t w[N];
  uint16_t s[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const auto [head, nb, is_v] = kv4_kind(c, blockIdx.y * N + n);
    w[n] = 0;
    s[n] = 0;
    if (blockIdx.y * N + n < kinds && at.page >= 0) {
      const char *base = page + (uint32_t)head * chunk;
      w[n] = ldg(reinterpret_cast<const uint32_t *>(base + (is_v ? ch.v_code(nb, at.at) : ch.k_code(nb, at.at)) + 4 * i));
      s[n] = ldg(reinterpret_cast<const uint16_t *>(base + (is_v ? ch.v_scale(nb, at.at) : ch.k_scale(nb, at.at))));
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (blockIdx.y * N + n >= kinds) break;
    const auto [head, nb, is_v] = kv4_kind(c, blockIdx.y * N + n);
    float x[8];
    kv4_values8(w[n], x);
    kv4_fwht16_signed(x, i);
    const float f = kv4_widen<true>(s[n]) * sign;
#pragma unroll
    for (int t = 0; t < 8; ++t) x[t] *= f;
    uint16_t *y = (is_v ? v : k) + ((size_t)row * c.n_kv_heads + head) * c.head_dim + nb * 128 + 8 * place;
    __builtin_nontemporal_store(kv4_pack8<BF>(x), reinterpret_cast<u32x4 *>(y));
  }
}

// ---------------------------------------------------------------------------------------
// Page operations
// ---------------------------------------------------------------------------------------
//
// Integers on a few kilobytes, then page bytes moved once.  One workgroup plans: it checks the
// call, sums what each item needs, finds the lowest free pages, and leaves a verdict, the items'
// first new page (an exclusive prefix sum) and the list of pages in the workspace, where the
// copying launch reads them.  A call that cannot be served whole changes nothing.

struct PagesPlan {
  int32_t *status;  // [0]: 1 = the call goes ahead
  int32_t *first;   // [n]: item i's new pages are list[first[i] ..]
  int32_t *list;    // [<= n_pages]
};

PagesPlan plan_of(void *ws, int n) {
  int32_t *p = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + kWsReserved);
  return PagesPlan{p, p + 64, p + 64 + (n + 63) / 64 * 64};
}

enum { kReserve = 0, kFork = 1, kCompact = 2 };

constexpr int kPlanThreads = 1024;

// Exclusive prefix sum over the workgroup's threads; *total gets the sum.  64-bit: a refused
// call's needs may add up to more than 2^31.  `lds`: 17 words.
__device__ __forceinline__ long long block_prefix(long long v, long long *lds, long long *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  long long x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long long y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  __syncthreads();  // (the last call's readers are done)
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
    long long s = 0;
    for (int w = 0; w < kPlanThreads / 64; ++w) {
      const long long t = lds[w];
      lds[w] = s;
      s += t;
    }
    lds[kPlanThreads / 64] = s;
  }
  __syncthreads();
  *total = lds[kPlanThreads / 64];
  return lds[wave] + x - v;
}

__device__ __forceinline__ int pages_of_len(int len, int T) { return (int)(((long long)len + T - 1) >> kv4_page_log2(T)); }

// What item i needs, or -1 where the call has to be refused.
template <int MODE>
__device__ int plan_need(const Kv4Pages &p, int i, const uint32_t *dst_bits) {
  const int T = p.c.page_size;
  const long long cap = (long long)p.max_pages * T;
  const int d = p.dst ? p.dst[i] : i;
  if ((uint32_t)d >= (uint32_t)p.n_slots) return -1;
  const int have = p.lens[d];
  if (have < 0 || have > cap) return -1;
  if (MODE == kReserve) {
    const int add = p.add[i];
    if (add < 0 || (long long)have + add > cap) return -1;
    return pages_of_len(have + add, T) - pages_of_len(have, T);
  }
  const int s = p.src[i];
  if ((uint32_t)s >= (uint32_t)p.n_slots) return -1;
  const int len = p.lens[s];
  if (len < 0 || len > cap) return -1;
  if (((dst_bits[s >> 5] >> (s & 31)) & 1) && !(MODE == kCompact && s == d)) return -1;  // a src that is written
  if (MODE == kFork) return len % T != 0;
  const int k0 = p.keep_cu[i], k1 = p.keep_cu[i + 1];
  if (k0 < 0 || k1 < k0 || k1 > p.n_keep || k1 - k0 > cap) return -1;
  return pages_of_len(k1 - k0, T);
}

template <int MODE>
__global__ __launch_bounds__(kPlanThreads) void kv4_plan_kernel(Kv4Pages p, PagesPlan plan, uint32_t *errword) {
  extern __shared__ uint32_t dst_bits[];  // one bit per slot
  __shared__ long long lds[kPlanThreads / 64 + 1];
  __shared__ int bad;
  const int tid = threadIdx.x;
  for (int w = tid; w < (p.n_slots + 31) / 32; w += kPlanThreads) dst_bits[w] = 0;
  if (tid == 0) bad = 0;
  __syncthreads();
  if (p.dst) {
    for (int i = tid; i < p.n; i += kPlanThreads) {
      const int d = p.dst[i];
      if ((uint32_t)d >= (uint32_t)p.n_slots) bad = 1;
      else if (atomicOr(&dst_bits[d >> 5], 1u << (d & 31)) >> (d & 31) & 1) bad = 1;  // named twice
    }
    __syncthreads();
  }
  long long need = 0;
  for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int want = i < p.n ? plan_need<MODE>(p, i, dst_bits) : 0;
    if (want < 0) bad = 1, want = 0;
    long long total;
    const long long before = block_prefix(want, lds, &total);
    if (i < p.n) plan.first[i] = (int)(need + before);
    need += total;
    if (need > p.c.n_pages) break;  // (uniform) more than there are
  }
  __syncthreads();
  if (bad || need > p.c.n_pages) {
    if (tid == 0) {
      plan.status[0] = 0;
      kv4_error(errword, bad ? TRELLIS_KV4_ERR_BAD : TRELLIS_KV4_ERR_NO_PAGES);
    }
    return;
  }
  // the lowest free pages, four per thread and round
  long long found = 0;
  for (int g0 = 0; g0 < p.c.n_pages && found < need; g0 += 4 * kPlanThreads) {
    const int g = g0 + 4 * tid;
    int is[4], n = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      is[t] = g + t < p.c.n_pages && p.ref[g + t] == 0;
      n += is[t];
    }
    long long total, at = found + block_prefix(n, lds, &total);
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (is[t]) {
        if (at < need) plan.list[at] = g + t;
        ++at;
      }
    found += total;
  }
  __syncthreads();  // the list is complete
  if (tid == 0) plan.status[0] = found >= need;
  if (found < need) {
    if (tid == 0) kv4_error(errword, TRELLIS_KV4_ERR_NO_PAGES);
    return;
  }
  if (MODE == kReserve) {  // nothing to copy: the same launch takes the pages, a wave an item
    const int T = p.c.page_size, lane = tid & 63;
    for (int i = tid >> 6; i < p.n; i += kPlanThreads / 64) {
      const int d = p.dst ? p.dst[i] : i;
      const int len = p.lens[d], now = len + p.add[i];
      const int h0 = pages_of_len(len, T), n = pages_of_len(now, T) - h0, first = plan.first[i];
      for (int j = lane; j < n; j += 64) {
        const int page = plan.list[first + j];
        p.table[(size_t)d * p.max_pages + h0 + j] = page;
        p.ref[page] = 1;
      }
      if (lane == 0) p.lens[d] = now;
    }
  }
}

// Drops one count of a slot's pages; `n` threads share the work, this one is thread t.
__device__ __forceinline__ void release_pages(const Kv4Pages &p, int slot, int len, int t, int n, uint32_t *errword) {
  const int count = pages_of_len(len, p.c.page_size);
  for (int j = t; j < count && j < p.max_pages; j += n) {
    const int page = p.table[(size_t)slot * p.max_pages + j];
    if ((uint32_t)page >= (uint32_t)p.c.n_pages) {
      kv4_error(errword, TRELLIS_KV4_ERR_BAD);
      continue;
    }
    if (atomicSub(&p.ref[page], 1) <= 0) {  // it was not held
      atomicAdd(&p.ref[page], 1);
      kv4_error(errword, TRELLIS_KV4_ERR_BAD);
    }
  }
}

// A child's table row and counts (workgroup y = 0), and its last page: a wave copies the rows that
// are filled of one (layer, head) at a time, codes and scales of keys and values together, so that
// up to 20 loads are in flight before the first store.  HBM bounds it (192 children of 48 parents, 32
// layers, 390 MB, and their release: 84 us); the stores bypass the caches, which keep the parents' pages
// where they are there already (59 us then, 126 with stores through the caches).
// Grid: x = item, y = shares of the (layer, head) units.
template <int NB>
__global__ __launch_bounds__(256) void kv4_fork_kernel(Kv4Pages p, PagesPlan plan, uint32_t *errword) {
  if (plan.status[0] != 1) return;
  const int i = blockIdx.x, T = p.c.page_size;
  const int s = p.src[i], d = p.dst[i], len = p.lens[s];
  const int full = len / T, part = len % T;
  const int32_t *from = p.table + (size_t)s * p.max_pages;
  if (blockIdx.y == 0) {
    __shared__ int old;
    if (threadIdx.x == 0) old = p.lens[d];
    __syncthreads();
    release_pages(p, d, old, threadIdx.x, 256, errword);
    __syncthreads();  // the old row is read
    int32_t *to = p.table + (size_t)d * p.max_pages;
    for (int j = threadIdx.x; j < full; j += 256) {
      const int page = from[j];
      to[j] = page;
      if ((uint32_t)page < (uint32_t)p.c.n_pages) atomicAdd(&p.ref[page], 1);
      else kv4_error(errword, TRELLIS_KV4_ERR_BAD);
    }
    if (threadIdx.x == 0) {
      if (part) {
        const int page = plan.list[plan.first[i]];
        to[full] = page;
        p.ref[page] = 1;
      }
      p.lens[d] = len;
    }
  }
  if (!part) return;
  const int a = from[full], z = plan.list[plan.first[i]];
  if ((uint32_t)a >= (uint32_t)p.c.n_pages) {
    if (blockIdx.y == 0 && threadIdx.x == 0) kv4_error(errword, TRELLIS_KV4_ERR_BAD);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int units = p.c.n_layers * p.c.n_kv_heads;
  for (int u = blockIdx.y * 4 + wave; u < units; u += gridDim.y * 4) {
    const int head = u % p.c.n_kv_heads, layer = u / p.c.n_kv_heads;
    const char *x = kv4_chunk(p.c, layer, a, head);
    char *y = kv4_chunk(p.c, layer, z, head);
    const char *xs = x + 128 * NB * T;
    char *ys = y + 128 * NB * T;
    for (int r0 = 0; r0 < part; r0 += 64) {  // 64 rows: four loads a part and a scale
      u32x4 v[2 * NB][4];
      uint16_t s[2 * NB];
#pragma unroll
      for (int q = 0; q < 2 * NB; ++q) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int o = r0 * 64 + k * 1024 + lane * 16;
          if (o < part * 64) v[q][k] = ldg(reinterpret_cast<const u32x4 *>(x + q * T * 64 + o));
        }
        if (r0 + lane < part) s[q] = ldg(reinterpret_cast<const uint16_t *>(xs + (q * T + r0 + lane) * 2));
      }
#pragma unroll
      for (int q = 0; q < 2 * NB; ++q) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int o = r0 * 64 + k * 1024 + lane * 16;
          if (o < part * 64) __builtin_nontemporal_store(v[q][k], reinterpret_cast<u32x4 *>(y + q * T * 64 + o));
        }
        if (r0 + lane < part) *reinterpret_cast<uint16_t *>(ys + (q * T + r0 + lane) * 2) = s[q];
      }
    }
  }
}

// Compaction's copy: a wave takes 16 kept rows (four lanes a row, 16 bytes a lane) and its share
// of the (layer, head, part) units, four at a time so that their loads are in flight together; a
// row's pages are looked up once for all units.  HBM bounds it: rows are 64 bytes, so where about half
// are kept most 128-byte lines are read for one of their two (12 x 55% of up to 4000 tokens, 16 layers:
// 300 MB kept, 174 us with ordinary accesses, 156 with ones that bypass the caches).
__global__ __launch_bounds__(256) void kv4_compact_copy_kernel(Kv4Pages p, PagesPlan plan, uint32_t *errword) {
  if (plan.status[0] != 1) return;
  const int T = p.c.page_size, log_t = kv4_page_log2(T), NB = p.c.head_dim >> 7;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = blockIdx.x * 16;
  __shared__ int4 rows[16];
  {  // 16 lanes find a row's item together
    const int group = threadIdx.x >> 4, row = r16 + group;
    int4 t = make_int4(-1, 0, -1, 0);  // page and place of the source, of the destination
    if (row < p.n_keep) {
      const int i = kv4_seq_of(p.keep_cu, p.n, row, threadIdx.x & 15);
      if (i < p.n && row >= p.keep_cu[i]) {
        const int s = p.src[i], pos = p.keep[row], j = row - p.keep_cu[i];
        if (pos >= 0 && pos < p.lens[s])
          t = make_int4(p.table[(size_t)s * p.max_pages + (pos >> log_t)], pos & (T - 1), plan.list[plan.first[i] + (j >> log_t)],
                        j & (T - 1));
      }
    }
    if ((threadIdx.x & 15) == 0) rows[group] = t;
  }
  __syncthreads();
  const int4 t = rows[lane >> 2];
  if ((uint32_t)t.x >= (uint32_t)p.c.n_pages || t.z < 0) {
    if (wave == 0 && blockIdx.y == 0 && (lane & 3) == 0 && r16 + (lane >> 2) < p.n_keep) kv4_error(errword, TRELLIS_KV4_ERR_BAD);
    return;
  }
  const int c = lane & 3, shift = NB == 1 ? 1 : 2;  // log2 of the parts
  const int units = (p.c.n_layers * p.c.n_kv_heads) << shift, stride = gridDim.y * 4;
  for (int u0 = blockIdx.y * 4 + wave; u0 < units; u0 += 4 * stride) {
    u32x4 v[4];
    uint16_t s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = u0 + k * stride, q = u & ((1 << shift) - 1), h = u >> shift;
      if (u < units) {
        const char *x = kv4_chunk(p.c, h / p.c.n_kv_heads, t.x, h % p.c.n_kv_heads);
        v[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(x + (q * T + t.y) * 64 + 16 * c));
        if (c == 0) s[k] = ldg(reinterpret_cast<const uint16_t *>(x + 128 * NB * T + (q * T + t.y) * 2));
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = u0 + k * stride, q = u & ((1 << shift) - 1), h = u >> shift;
      if (u < units) {
        char *y = kv4_chunk(p.c, h / p.c.n_kv_heads, t.z, h % p.c.n_kv_heads);
        __builtin_nontemporal_store(v[k], reinterpret_cast<u32x4 *>(y + (q * T + t.w) * 64 + 16 * c));
        if (c == 0) *reinterpret_cast<uint16_t *>(y + 128 * NB * T + (q * T + t.w) * 2) = s[k];
      }
    }
  }
}

// Compaction's tables, once every row is copied (dst may be the src).
__global__ __launch_bounds__(256) void kv4_compact_commit_kernel(Kv4Pages p, PagesPlan plan, uint32_t *errword) {
  if (plan.status[0] != 1) return;
  const int i = blockIdx.x, d = p.dst[i];
  __shared__ int old;
  if (threadIdx.x == 0) old = p.lens[d];
  __syncthreads();
  release_pages(p, d, old, threadIdx.x, 256, errword);
  __syncthreads();  // the old row is read
  const int kept = p.keep_cu[i + 1] - p.keep_cu[i], count = pages_of_len(kept, p.c.page_size), first = plan.first[i];
  for (int j = threadIdx.x; j < count; j += 256) {
    const int page = plan.list[first + j];
    p.table[(size_t)d * p.max_pages + j] = page;
    p.ref[page] = 1;
  }
  if (threadIdx.x == 0) p.lens[d] = kept;
}

// Every workgroup checks the whole list before it releases its slots: what another one has released by
// then is a length of zero, which is in range, so all of them come to the same verdict.
__global__ __launch_bounds__(256) void kv4_free_kernel(Kv4Pages p, uint32_t *errword) {
  __shared__ int bad, len;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  const long long cap = (long long)p.max_pages * p.c.page_size;
#pragma unroll 4
  for (int i = threadIdx.x; i < p.n; i += 256) {
    const int d = p.dst[i];
    const bool ok = (uint32_t)d < (uint32_t)p.n_slots;
    const int l = ok ? p.lens[d] : -1;
    if (l < 0 || l > cap) bad = 1;
  }
  __syncthreads();
  if (bad) {
    if (blockIdx.x == 0 && threadIdx.x == 0) kv4_error(errword, TRELLIS_KV4_ERR_BAD);
    return;
  }
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int d = p.dst[i];
    if (threadIdx.x == 0) len = atomicExch(&p.lens[d], 0);  // a slot named twice is empty the second time
    __syncthreads();
    release_pages(p, d, len, threadIdx.x, 256, errword);
    __syncthreads();  // len is read
  }
}

size_t bits_bytes(int n_slots) { return (size_t)((n_slots + 31) / 32) * 4; }

}  // namespace

namespace {
// Kinds a workgroup takes: four where 2048 workgroups (eight a CU) remain.
int kinds_each(const trellis_kv4_cache &c, const trellis_kv4_batch &b) {
  const long long groups = (long long)((b.rows + 15) / 16) * 2 * c.n_kv_heads * (c.head_dim / 128);
  return groups >= 4 * 2048 ? 4 : 1;
}
}  // namespace

hipError_t launch_kv4_append(const trellis_kv4_cache &c, int layer, const trellis_kv4_batch &b, int dtype,
                             const Kv4Rows &k, const Kv4Rows &v, uint32_t *errword, hipStream_t stream) {
  const int n = kinds_each(c, b), kinds = 2 * c.n_kv_heads * (c.head_dim / 128);
  const dim3 grid((b.rows + 15) / 16, (kinds + n - 1) / n);
  const bool bf = dtype == TRELLIS_KV4_BF16;
  const auto kernel = n == 4 ? (bf ? kv4_append_kernel<true, 4> : kv4_append_kernel<false, 4>)
                             : (bf ? kv4_append_kernel<true, 1> : kv4_append_kernel<false, 1>);
  kernel<<<grid, 256, 0, stream>>>(c, layer, b, k, v, errword);
  return hipGetLastError();
}

hipError_t launch_kv4_read(const trellis_kv4_cache &c, int layer, const trellis_kv4_batch &b, int dtype, void *k,
                           void *v, uint32_t *errword, hipStream_t stream) {
  const int n = kinds_each(c, b), kinds = 2 * c.n_kv_heads * (c.head_dim / 128);
  const dim3 grid((b.rows + 15) / 16, (kinds + n - 1) / n);
  const bool bf = dtype == TRELLIS_KV4_BF16;
  const auto kernel = n == 4 ? (bf ? kv4_read_kernel<true, 4> : kv4_read_kernel<false, 4>)
                             : (bf ? kv4_read_kernel<true, 1> : kv4_read_kernel<false, 1>);
  kernel<<<grid, 256, 0, stream>>>(c, layer, b, static_cast<uint16_t *>(k), static_cast<uint16_t *>(v), errword);
  return hipGetLastError();
}

size_t kv4_pages_workspace_bytes(int n_pages, int n) {
  return kWsReserved + 256 + (size_t)(n + 63) / 64 * 256 + (size_t)n_pages * 4;
}

hipError_t launch_kv4_reserve(const Kv4Pages &p, void *ws, hipStream_t stream) {
  kv4_plan_kernel<kReserve><<<1, kPlanThreads, bits_bytes(p.n_slots), stream>>>(p, plan_of(ws, p.n), static_cast<uint32_t *>(ws));
  return hipGetLastError();
}

hipError_t launch_kv4_fork(const Kv4Pages &p, void *ws, hipStream_t stream) {
  const PagesPlan plan = plan_of(ws, p.n);
  uint32_t *err = static_cast<uint32_t *>(ws);
  kv4_plan_kernel<kFork><<<1, kPlanThreads, bits_bytes(p.n_slots), stream>>>(p, plan, err);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const int units = p.c.n_layers * p.c.n_kv_heads;
  const dim3 grid(p.n, (units + 3) / 4 < 4096 ? (units + 3) / 4 : 4096);
  if (p.c.head_dim == 128) kv4_fork_kernel<1><<<grid, 256, 0, stream>>>(p, plan, err);
  else kv4_fork_kernel<2><<<grid, 256, 0, stream>>>(p, plan, err);
  return hipGetLastError();
}

hipError_t launch_kv4_compact(const Kv4Pages &p, void *ws, hipStream_t stream) {
  const PagesPlan plan = plan_of(ws, p.n);
  uint32_t *err = static_cast<uint32_t *>(ws);
  kv4_plan_kernel<kCompact><<<1, kPlanThreads, bits_bytes(p.n_slots), stream>>>(p, plan, err);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (p.n_keep > 0) {
    const int units = p.c.n_layers * p.c.n_kv_heads * 2 * (p.c.head_dim / 128);
    const int y = (units + 15) / 16;
    kv4_compact_copy_kernel<<<dim3((p.n_keep + 15) / 16, y < 1024 ? y : 1024), 256, 0, stream>>>(p, plan, err);
    // (the tables must not change to pages that nothing filled)
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  kv4_compact_commit_kernel<<<p.n, 256, 0, stream>>>(p, plan, err);
  return hipGetLastError();
}

hipError_t launch_kv4_free(const Kv4Pages &p, uint32_t *errword, hipStream_t stream) {
  kv4_free_kernel<<<p.n < 1024 ? p.n : 1024, 256, 0, stream>>>(p, errword);
  return hipGetLastError();
}

}  // namespace trellis
