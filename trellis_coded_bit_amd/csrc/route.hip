// Tokens sorted by expert and back (include/trellis_route.h).
//
// Sort: a counting sort that keeps the order of equal ids.  A workgroup takes 1024 entries, one a
// thread.  An entry's position is: the entries of smaller ids (a scan of all counts), those of its
// id in earlier workgroups' entries, in earlier waves, and in earlier lanes (ballots).
#include "f8_device.h"

namespace trellis {

namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
// Entries up to which every workgroup counts all of them itself; above, a launch before counts.
constexpr int kSortOne = 1 << 16;

// The id as a key: what is not here counts as one more expert behind the others.
__device__ __forceinline__ int sort_key(const int32_t *ids, long long i, int E, uint32_t *errword) {
  const int id = ldg(ids + i);
  if (id >= 0 && id < E) return id;
  if (id != -1) f8_error(errword);
  return E;
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int32_t *ids, int n, int E, uint32_t *counts,
                                                                  uint32_t *errword) {
  extern __shared__ uint32_t c[];  // [E + 1]
  for (int e = threadIdx.x; e <= E; e += kSortThreads) c[e] = 0;
  __syncthreads();
  const long long i = (long long)blockIdx.x * kSortThreads + threadIdx.x;
  if (i < n) atomicAdd(&c[sort_key(ids, i, E, errword)], 1u);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kSortThreads) counts[(size_t)blockIdx.x * (E + 1) + e] = c[e];
}

// counts: NULL, or [workgroups][E + 1] from the launch before.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const int32_t *ids, int n, int E, int id_bits,
                                                                  const uint32_t *counts, int32_t *offsets, int32_t *order,
                                                                  int32_t *inverse, uint32_t *errword) {
  extern __shared__ uint32_t lds[];
  uint32_t *before = lds;                // [E + 1] of the id in earlier workgroups' entries, then its first position here
  uint32_t *all = before + E + 1;        // [E + 1] of the id at all
  uint16_t *waves = reinterpret_cast<uint16_t *>(all + E + 1);  // [16][E + 1] of the id in this workgroup's waves
  __shared__ uint32_t sums[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e <= E; e += kSortThreads) before[e] = all[e] = 0;
  for (int e = tid; e < kSortWaves * (E + 1); e += kSortThreads) waves[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * kSortThreads;
  if (counts) {
    for (int e = tid; e <= E; e += kSortThreads) {
      uint32_t b = 0, t = 0;
      for (int g = 0; g < (int)gridDim.x; ++g) {
        const uint32_t c = ldg(counts + (size_t)g * (E + 1) + e);
        t += c;
        if (g < (int)blockIdx.x) b += c;
      }
      before[e] = b;
      all[e] = t;
    }
  } else {
    for (int i = tid; i < n; i += kSortThreads) {
      const int key = sort_key(ids, i, E, errword);
      atomicAdd(&all[key], 1u);
      if (i < first) atomicAdd(&before[key], 1u);
    }
  }
  // the lanes of the wave with the same key
  const int i = first + tid;
  const bool live = i < n;
  const int key = live ? sort_key(ids, i, E, errword) : E;
  uint64_t same = __ballot(live);
  for (int b = 0; b < id_bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    same &= ((key >> b) & 1) ? set : ~set;
  }
  const int rank = __popcll(same & ((1ull << lane) - 1));
  if (live && rank == 0) waves[wave * (E + 1) + key] = (uint16_t)__popcll(same);
  __syncthreads();
  // exclusive scan of all counts over the ids, 1024 at a time
  uint32_t carry = 0;
  for (int e0 = 0; e0 <= E; e0 += kSortThreads) {
    const int e = e0 + tid;
    const uint32_t c = e <= E ? all[e] : 0;
    uint32_t s = c;
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(s, d, 64);
      if (lane >= d) s += o;
    }
    if (lane == 63) sums[wave] = s;
    __syncthreads();
    uint32_t base = carry;
    for (int w = 0; w < kSortWaves; ++w) {
      if (w < wave) base += sums[w];
      carry += sums[w];
    }
    if (e <= E) {
      const uint32_t start = base + s - c;
      before[e] += start;
      if (blockIdx.x == 0) offsets[e] = (int32_t)start;
    }
    __syncthreads();
  }
  if (!live) return;
  uint32_t pos = before[key] + rank;
  for (int w = 0; w < wave; ++w) pos += waves[w * (E + 1) + key];
  const bool here = key < E;
  inverse[i] = here ? (int32_t)pos : -1;
  order[pos] = here ? i : -1;
}

size_t sort_lds(int E) { return (size_t)(E + 1) * (4 + 4 + 2 * kSortWaves); }

template <typename T>
__global__ __launch_bounds__(256) void gather_kernel(const char *x, int64_t x_row, int tokens, int64_t row_words,
                                                     const int32_t *order, int rows, int per, int parts, T *out,
                                                     uint32_t *errword) {
  const long long items = (long long)rows * parts;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int row = (int)(it / parts), part = (int)(it - (long long)row * parts);
    const int entry = ldg(order + row);
    if (entry == -1) continue;
    if (entry < 0 || entry / per >= tokens) {
      if (threadIdx.x == 0) f8_error(errword);
      continue;
    }
    const int64_t w = (int64_t)part * 256 + threadIdx.x;
    if (w < row_words) stg(out + row * row_words + w, ldg(reinterpret_cast<const T *>(x + (entry / per) * x_row) + w));
  }
}

template <bool BF>
__global__ __launch_bounds__(256) void combine_kernel(MoeCombine a, int parts, uint32_t *errword) {
  const long long items = (long long)a.tokens * parts;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int t = (int)(it / parts), part = (int)(it - (long long)t * parts);
    const int c = (part * 256 + threadIdx.x) * 8;
    if (c >= a.n) continue;
    float s[8] = {};
    if (a.add) f8_widen8<BF>(ldg(reinterpret_cast<const u32x4 *>(a.add + (size_t)t * a.n + c)), s);
    for (int j = 0; j < a.top; ++j) {
      const int pos = ldg(a.inverse + (size_t)t * a.top + j);
      if (pos == -1) continue;
      if ((uint32_t)pos >= (uint32_t)a.rows) {
        f8_error(errword);
        continue;
      }
      const float w = a.weights ? ldg(a.weights + (size_t)t * a.top + j) : 1.f;
      float v[8];
      f8_widen8<BF>(ldg(reinterpret_cast<const u32x4 *>(a.y + (size_t)pos * a.n + c)), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = fmaf(w, v[i], s[i]);
    }
    stg(reinterpret_cast<u32x4 *>(a.out + (size_t)t * a.n + c), f8_narrow8<BF>(s));
  }
}

// A workgroup a token; its choices eight at a time, so that d_out is read once for them.
template <bool BF>
__global__ __launch_bounds__(256) void combine_grad_kernel(MoeCombine a, uint32_t *errword) {
  __shared__ float part[4][8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    for (int j0 = 0; j0 < a.top; j0 += 8) {
      int pos[8];
      float w[8], dot[8] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        pos[j] = -1;
        w[j] = 1.f;
        if (j0 + j < a.top) {
          pos[j] = ldg(a.inverse + (size_t)t * a.top + j0 + j);
          if (a.weights) w[j] = ldg(a.weights + (size_t)t * a.top + j0 + j);
        }
        if (pos[j] != -1 && (uint32_t)pos[j] >= (uint32_t)a.rows) {
          f8_error(errword);
          pos[j] = -1;
        }
      }
      for (int c = threadIdx.x * 8; c < a.n; c += 256 * 8) {
        float d[8];
        f8_widen8<BF>(ldg(reinterpret_cast<const u32x4 *>(a.d_out + (size_t)t * a.n + c)), d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (pos[j] < 0) continue;
          const size_t at = (size_t)pos[j] * a.n + c;
          if (a.d_weights) {
            float v[8];
            f8_widen8<BF>(ldg(reinterpret_cast<const u32x4 *>(a.y + at)), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[j] = fmaf(d[i], v[i], dot[j]);
          }
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = w[j] * d[i];
          stg(reinterpret_cast<u32x4 *>(a.out + at), f8_narrow8<BF>(o));
        }
      }
      if (!a.d_weights) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = dot[j];
        v += lane_xor<1>(v);
        v += lane_xor<2>(v);
        v += lane_xor<4>(v);
        v += lane_xor<8>(v);
        v += lane_xor<16>(v);
        v += lane_xor<32>(v);
        if (lane == 0) part[wave][j] = v;
      }
      __syncthreads();
      if (threadIdx.x < 8 && j0 + (int)threadIdx.x < a.top)
        a.d_weights[(size_t)t * a.top + j0 + threadIdx.x] =
            (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
      __syncthreads();
    }
  }
}

unsigned grid_of(long long items) { return (unsigned)(items < (1 << 22) ? items : (1 << 22)); }

}  // namespace

size_t moe_sort_workspace_bytes(int tokens, int top, int n_experts) {
  const long long n = (long long)tokens * top;
  if (n <= kSortOne) return kWsReserved;
  return kWsReserved + (size_t)((n + kSortThreads - 1) / kSortThreads) * (n_experts + 1) * 4;
}

hipError_t launch_moe_sort(const int32_t *ids, int tokens, int top, int n_experts, int32_t *offsets, int32_t *order,
                           int32_t *inverse, void *ws, hipStream_t stream) {
  const int n = tokens * top;
  const int grid = n ? (n + kSortThreads - 1) / kSortThreads : 1;
  uint32_t *errword = static_cast<uint32_t *>(ws), *counts = nullptr;
  int bits = 1;
  while ((1 << bits) <= n_experts) ++bits;  // keys 0 .. n_experts
  const size_t lds = sort_lds(n_experts);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(sort_place_kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  if (n > kSortOne) {
    counts = reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + kWsReserved);
    sort_count_kernel<<<grid, kSortThreads, (n_experts + 1) * 4, stream>>>(ids, n, n_experts, counts, errword);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  sort_place_kernel<<<grid, kSortThreads, lds, stream>>>(ids, n, n_experts, bits, counts, offsets, order, inverse, errword);
  return hipGetLastError();
}

hipError_t launch_moe_gather(const void *x, int64_t x_row_bytes, int tokens, int64_t row_bytes, const int32_t *order,
                             int rows, int per, void *out, uint32_t *errword, hipStream_t stream) {
  const char *p = static_cast<const char *>(x);
  const bool wide = row_bytes % 16 == 0 && x_row_bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(x) % 16) == 0 &&
                    (reinterpret_cast<uintptr_t>(out) % 16) == 0;
  const int64_t words = row_bytes / (wide ? 16 : 4);
  const int parts = (int)((words + 255) / 256);
  const unsigned grid = grid_of((long long)rows * parts);
  if (wide) gather_kernel<u32x4><<<grid, 256, 0, stream>>>(p, x_row_bytes, tokens, words, order, rows, per, parts, static_cast<u32x4 *>(out), errword);
  else gather_kernel<uint32_t><<<grid, 256, 0, stream>>>(p, x_row_bytes, tokens, words, order, rows, per, parts, static_cast<uint32_t *>(out), errword);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombine &a, uint32_t *errword, hipStream_t stream) {
  const int parts = (a.n / 8 + 255) / 256;
  const unsigned grid = grid_of((long long)a.tokens * parts);
  if (a.bf16) combine_kernel<true><<<grid, 256, 0, stream>>>(a, parts, errword);
  else combine_kernel<false><<<grid, 256, 0, stream>>>(a, parts, errword);
  return hipGetLastError();
}

hipError_t launch_moe_combine_grad(const MoeCombine &a, uint32_t *errword, hipStream_t stream) {
  const unsigned grid = grid_of(a.tokens);
  if (a.bf16) combine_grad_kernel<true><<<grid, 256, 0, stream>>>(a, errword);
  else combine_grad_kernel<false><<<grid, 256, 0, stream>>>(a, errword);
  return hipGetLastError();
}

}  // namespace trellis
