// Tokens sorted by expert and back (include/trellis_route.h).
//
// Sort: a counting sort that keeps the order of equal ids.  A workgroup places 1024 entries, one a
// thread.  An entry's position is: the entries of smaller ids (a scan of all counts), those of its
// id in earlier workgroups' entries, in earlier waves, and in earlier lanes (ballots).  Up to 65536
// entries every workgroup counts all of them itself, in one launch, with up to 64 ids a thread (us with
// one | three launches: 4000 entries 6.5 | 10.9, 32768 7.6 | 10.8, 65536 10.7 | 10.9, 131072 17.1 |
// 10.8).  Above, two launches before count and scan.  All of it is latency: of 264 entries 3.9 us in
// the kernel, of 32776 8.3.
//
// Gather, combine and gradient move rows and are bound by memory: what each has to read and write at
// a copy's 5 TB/s is given at the kernel.
#include "f8_device.h"

namespace trellis {

namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortOne = 1 << 16;

// An id, or -1 for an expert that is not here.
__device__ __forceinline__ int sort_key(int id, int E, uint32_t *errword) {
  if (id >= 0 && id < E) return id;
  if (id != -1) f8_error(errword);
  return -1;
}

// counts [E][groups]: of each id in each workgroup's entries.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int32_t *ids, int n, int E, uint32_t *counts) {
  extern __shared__ uint32_t c[];  // [E]
  for (int e = threadIdx.x; e < E; e += kSortThreads) c[e] = 0;
  __syncthreads();
  const int i = blockIdx.x * kSortThreads + threadIdx.x;
  const int id = i < n ? ldg(ids + i) : -1;
  if (id >= 0 && id < E) atomicAdd(&c[id], 1u);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) counts[(size_t)e * gridDim.x + blockIdx.x] = c[e];
}

// A workgroup an id: its counts become the sums before them, its total goes to totals.
__global__ __launch_bounds__(256) void sort_scan_kernel(uint32_t *counts, int groups, uint32_t *totals) {
  __shared__ uint32_t sums[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t *row = counts + (size_t)blockIdx.x * groups, carry = 0;
  for (int g0 = 0; g0 < groups; g0 += 256) {
    const int g = g0 + threadIdx.x;
    const uint32_t c = g < groups ? row[g] : 0;
    uint32_t s = c;
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(s, d, 64);
      if (lane >= d) s += o;
    }
    if (lane == 63) sums[wave] = s;
    __syncthreads();
    uint32_t base = carry;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) base += sums[w];
      carry += sums[w];
    }
    if (g < groups) row[g] = base + s - c;
    __syncthreads();
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// counts: NULL, or the sums and totals of the launches before.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const int32_t *ids, int n, int E, int id_bits,
                                                                  const uint32_t *counts, const uint32_t *totals,
                                                                  int32_t *offsets, int32_t *order, int32_t *inverse,
                                                                  uint32_t *errword) {
  extern __shared__ uint32_t lds[];
  uint32_t *before = lds;       // [E] of the id in earlier workgroups' entries, then its first position here
  uint32_t *after = before + E; // [E] of the id in the others
  uint16_t *waves = reinterpret_cast<uint16_t *>(after + E);  // [16][E] of the id in this workgroup's waves
  __shared__ uint32_t sums[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int first = blockIdx.x * kSortThreads;
  const int i = first + tid;
  const int key = i < n ? sort_key(ldg(ids + i), E, errword) : -1;
  for (int e = tid; e < E; e += kSortThreads) {
    before[e] = counts ? ldg(counts + (size_t)e * gridDim.x + blockIdx.x) : 0;
    after[e] = counts ? ldg(totals + e) - before[e] : 0;
  }
  for (int e = tid; e < kSortWaves * E; e += kSortThreads) waves[e] = 0;
  __syncthreads();
  if (!counts) {
    // (what is not here is not counted: its entries need no position)
    for (int k0 = tid; k0 < n; k0 += 8 * kSortThreads) {
      int id[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) id[k] = k0 + k * kSortThreads < n ? ldg(ids + k0 + k * kSortThreads) : -1;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (id[k] >= 0 && id[k] < E) atomicAdd((k0 + k * kSortThreads < first ? before : after) + id[k], 1u);
    }
  }
  // the lanes of the wave with the same key
  uint64_t same = __ballot(key >= 0);
  for (int b = 0; b < id_bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    same &= ((key >> b) & 1) ? set : ~set;
  }
  const int rank = __popcll(same & ((1ull << lane) - 1));
  if (key >= 0 && rank == 0) waves[wave * E + key] = (uint16_t)__popcll(same);
  __syncthreads();
  // exclusive scan of all counts over the ids, 1024 at a time
  uint32_t carry = 0;
  for (int e0 = 0; e0 < E; e0 += kSortThreads) {
    const int e = e0 + tid;
    const uint32_t c = e < E ? before[e] + after[e] : 0;
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
    if (e < E) {
      const uint32_t start = base + s - c;
      before[e] += start;
      if (blockIdx.x == 0) offsets[e] = (int32_t)start;
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) offsets[E] = (int32_t)carry;
  if (i >= n) return;
  if ((uint32_t)i >= carry) order[i] = -1;  // (positions behind the last are nobody's)
  int32_t pos = -1;
  if (key >= 0) {
    uint32_t at = before[key] + rank;
    for (int w = 0; w < wave; ++w) at += waves[w * E + key];
    // (below n, unless the ids change while they are read, or another call writes the counts)
    if (at < (uint32_t)n) {
      pos = (int32_t)at;
      order[pos] = i;
    }
  }
  inverse[i] = pos;
}

// What sort_place_kernel has in shared memory besides its waves' sums.  (Those at the end of it, where
// their place is not a constant: 33 tokens' 264 entries 4.4 us for 3.75, 32776 entries 8.0 for 7.35.)
size_t sort_lds(int E) { return (size_t)E * (4 + 4 + 2 * kSortWaves); }

// A workgroup a row, four words a thread under way.  16411 rows of 6144 16-bit channels (252 MB moved at
// most, a token's row up to four times from a cache): 62 us; one word a thread: 78.
template <typename T, bool NT>
__global__ __launch_bounds__(256) void gather_kernel(const char *x, int64_t x_row, int tokens, int64_t row_words,
                                                     const int32_t *order, int rows, int per, T *out, uint32_t *errword) {
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    const int entry = ldg(order + row);
    if (entry == -1) continue;
    if (entry < 0 || entry / per >= tokens) {
      if (threadIdx.x == 0) f8_error(errword);
      continue;
    }
    const T *from = reinterpret_cast<const T *>(x + (entry / per) * x_row);
    T *to = out + row * row_words;
    for (int64_t w = threadIdx.x; w < row_words; w += 1024) {
      T v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (w + 256 * k < row_words) v[k] = ldg(from + w + 256 * k);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (w + 256 * k < row_words) stg_once<NT>(to + w + 256 * k, v[k]);
    }
  }
}

// Eight columns a thread, 2048 of a token a workgroup; a token's rows eight at a time, all under way before
// one is added.  The entries without a position are left out first: nothing of theirs is read.  4097
// tokens of 6144 channels with half of 8 entries here (252 MB): 43 us, as a copy; row after row with cached
// reads it took 95.  (All of a token's columns by one workgroup, one after the other, in us for the time
// here: 256 tokens of 8 with 6144 channels 8.8 for 7.8, 4096 with 5120 channels 72.9 for 69.5, 2048 with
// 20480 143 for 130; never less by more than 2 %.)
template <bool BF, bool NT>
__global__ __launch_bounds__(256) void combine_kernel(MoeCombine a, int groups, uint32_t *errword) {
  const int lane = threadIdx.x & 63;
  const long long items = (long long)a.tokens * groups;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int t = (int)(it / groups), c0 = (int)(it - (long long)t * groups) * 2048, c = c0 + threadIdx.x * 8;
    const bool live = c < a.n;
    const int at = live ? c : c0;
    float s[8] = {};
    u32x4 add = {0, 0, 0, 0};
    if (a.add) add = ldg(reinterpret_cast<const u32x4 *>(a.add + (size_t)t * a.n + at));
    bool first = true;
    for (int j0 = 0; j0 < a.top; j0 += 64) {
      int pos = -1;
      float weight = 1.f;
      if (j0 + lane < a.top) {
        pos = ldg(a.inverse + (size_t)t * a.top + j0 + lane);
        if (a.weights) weight = ldg(a.weights + (size_t)t * a.top + j0 + lane);
      }
      if (pos != -1 && (uint32_t)pos >= (uint32_t)a.rows) {
        f8_error(errword);
        pos = -1;
      }
      uint64_t left = __ballot(pos >= 0);
      while (left) {
        u32x4 v[8];
        float w[8];
        int count = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (!left) break;
          const int l = __builtin_ctzll(left);
          left &= left - 1;
          w[k] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), l));
          v[k] = ldg_once<NT>(reinterpret_cast<const u32x4 *>(a.y + (size_t)__builtin_amdgcn_readlane(pos, l) * a.n + at));
          ++count;
        }
        if (first && a.add) f8_widen8<BF>(add, s);
        first = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k >= count) break;
          float x[8];
          f8_widen8<BF>(v[k], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = fmaf(w[k], x[i], s[i]);
        }
      }
    }
    if (first && a.add) f8_widen8<BF>(add, s);
    if (live) stg(reinterpret_cast<u32x4 *>(a.out + (size_t)t * a.n + c), f8_narrow8<BF>(s));
  }
}

// A workgroup a token; its choices eight at a time, so that d_out is read once for them.  A weight's
// gradient is a chain of fmas a thread, then a tree over the workgroup: the same sum every time.  4096
// tokens of 8 with 5120 channels (713 MB): 143 us, a copy's rate.
template <bool BF, bool NT>
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
            f8_widen8<BF>(ldg_once<NT>(reinterpret_cast<const u32x4 *>(a.y + at)), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[j] = fmaf(d[i], v[i], dot[j]);
          }
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = w[j] * d[i];
          stg_once<NT>(reinterpret_cast<u32x4 *>(a.out + at), f8_narrow8<BF>(o));
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
  return kWsReserved + ((size_t)(n + kSortThreads - 1) / kSortThreads + 1) * n_experts * 4;
}

hipError_t launch_moe_sort(const int32_t *ids, int tokens, int top, int n_experts, int32_t *offsets, int32_t *order,
                           int32_t *inverse, void *ws, hipStream_t stream) {
  const int n = tokens * top;
  const int grid = n ? (n + kSortThreads - 1) / kSortThreads : 1;
  uint32_t *errword = static_cast<uint32_t *>(ws), *counts = nullptr, *totals = nullptr;
  int bits = 1;
  while ((1 << bits) < n_experts) ++bits;
  const size_t lds = sort_lds(n_experts);
  hipError_t e;
  if (lds + 4 * kSortWaves > 65536) {
    // (the most of any call: another thread's may be between this and its launch)
    e = hipFuncSetAttribute(reinterpret_cast<const void *>(sort_place_kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)sort_lds(kMoeExperts));
    if (e != hipSuccess) return e;
  }
  if (n > kSortOne) {
    counts = reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + kWsReserved);
    totals = counts + (size_t)grid * n_experts;
    sort_count_kernel<<<grid, kSortThreads, n_experts * 4, stream>>>(ids, n, n_experts, counts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    sort_scan_kernel<<<n_experts, 256, 0, stream>>>(counts, grid, totals);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  sort_place_kernel<<<grid, kSortThreads, lds, stream>>>(ids, n, n_experts, bits, counts, totals, offsets, order, inverse, errword);
  return hipGetLastError();
}

hipError_t launch_moe_gather(const void *x, int64_t x_row_bytes, int tokens, int64_t row_bytes, const int32_t *order,
                             int rows, int per, void *out, uint32_t *errword, hipStream_t stream) {
  const char *p = static_cast<const char *>(x);
  const bool wide = row_bytes % 16 == 0 && x_row_bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(x) % 16) == 0 &&
                    (reinterpret_cast<uintptr_t>(out) % 16) == 0;
  const int64_t words = row_bytes / (wide ? 16 : 4);
  const unsigned grid = grid_of(rows);
  const bool once = (size_t)rows * row_bytes > kF8Once;
  if (wide && once) gather_kernel<u32x4, true><<<grid, 256, 0, stream>>>(p, x_row_bytes, tokens, words, order, rows, per, static_cast<u32x4 *>(out), errword);
  else if (wide) gather_kernel<u32x4, false><<<grid, 256, 0, stream>>>(p, x_row_bytes, tokens, words, order, rows, per, static_cast<u32x4 *>(out), errword);
  else gather_kernel<uint32_t, false><<<grid, 256, 0, stream>>>(p, x_row_bytes, tokens, words, order, rows, per, static_cast<uint32_t *>(out), errword);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombine &a, uint32_t *errword, hipStream_t stream) {
  const int groups = (a.n + 2047) / 2048;
  const unsigned grid = grid_of((long long)a.tokens * groups);
  const bool once = (size_t)a.rows * a.n * 2 > kF8Once;
  if (a.bf16 && once) combine_kernel<true, true><<<grid, 256, 0, stream>>>(a, groups, errword);
  else if (a.bf16) combine_kernel<true, false><<<grid, 256, 0, stream>>>(a, groups, errword);
  else if (once) combine_kernel<false, true><<<grid, 256, 0, stream>>>(a, groups, errword);
  else combine_kernel<false, false><<<grid, 256, 0, stream>>>(a, groups, errword);
  return hipGetLastError();
}

hipError_t launch_moe_combine_grad(const MoeCombine &a, uint32_t *errword, hipStream_t stream) {
  const unsigned grid = grid_of(a.tokens);
  const bool once = (size_t)a.rows * a.n * 2 > kF8Once;
  if (a.bf16 && once) combine_grad_kernel<true, true><<<grid, 256, 0, stream>>>(a, errword);
  else if (a.bf16) combine_grad_kernel<true, false><<<grid, 256, 0, stream>>>(a, errword);
  else if (once) combine_grad_kernel<false, true><<<grid, 256, 0, stream>>>(a, errword);
  else combine_grad_kernel<false, false><<<grid, 256, 0, stream>>>(a, errword);
  return hipGetLastError();
}

}  // namespace trellis
