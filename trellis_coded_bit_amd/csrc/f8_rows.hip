// Row operators with a block-scaled E4M3 result: the norm with the residual's addition and the
// gated activation (include/trellis_f8.h).
//
// Eight channels a lane (16 bytes in, 8 out), so the 16 lanes of a DPP row hold a block of 128 and
// find its largest magnitude without shared memory.
#include "f8_device.h"

namespace trellis {

namespace {

// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += lane_xor<1>(v);
  v += lane_xor<2>(v);
  v += lane_xor<4>(v);
  v += lane_xor<8>(v);
  v += lane_xor<16>(v);
  v += lane_xor<32>(v);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// Sum over the workgroup, in every thread; `part` has a place for each of its waves.
template <typename T>
__device__ __forceinline__ T group_sum(T v, T *part) {
  v = wave_sum(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < waves; ++w) v += part[w];
  return v;
}

template <bool BF>
__device__ __forceinline__ void put_block(const F8RowsOut &o, const float (&u)[8], float post, bool live, size_t row, int n,
                                          int chunk) {
  if (o.q) {
    const F8Scale f = f8_scale(row16_umax(live ? magnitude8(u) : 0u), post);
    if (live) {
      stg(reinterpret_cast<u32x2 *>(o.q + row * n + 8 * chunk), f8_codes(u, f.inv));
      if ((chunk & 15) == 0) stg(o.scale + row * ((n + 127) >> 7) + (chunk >> 4), f.scale);
    }
  }
  if (o.y && live) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u[i] * post;
    stg(reinterpret_cast<u32x4 *>(o.y + row * n + 8 * chunk), f8_narrow8<BF>(v));
  }
}

// A workgroup a row, V chunks of eight channels a thread, held in registers from the one read to
// the results.  The row's factor 1 / sqrt(mean + eps) does not change which codes a block gets, so
// codes are made of u = h * gamma and the factor goes into the scale.  Where f32 does not hold the
// square sum or a block's u (bf16 reaches 3e38), they are formed in 64 bits instead.  Sums and u are f32
// and rounded once, to E4M3 or 16 bits; h is rounded only for h_out, not for the norm.
// 4097 rows of 6144 with a residual (177 MB): 30 us, 5.9 TB/s.  One row of 5120: 3.1 us, latency.
template <bool BF, int V>
__global__ __launch_bounds__(1024) void norm_kernel(F8Norm a) {
  __shared__ float part[16];
  __shared__ double part64[16];
  const size_t row = blockIdx.x;
  const int chunks = a.n >> 3;
  float h[V][8];
  u32x4 xs[V], rs[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = min(threadIdx.x + k * blockDim.x, (uint32_t)chunks - 1);
    xs[k] = ldg(reinterpret_cast<const u32x4 *>(a.x + row * a.x_row) + c);
    if (a.residual) rs[k] = ldg(reinterpret_cast<const u32x4 *>(a.residual + row * a.n) + c);
  }
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
    f8_widen8<BF>(xs[k], h[k]);
    if (a.residual) {
      float r[8];
      f8_widen8<BF>(rs[k], r);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] += r[i];
    }
    if (c < chunks) {
      if (a.h) stg(reinterpret_cast<u32x4 *>(a.h + row * a.n) + c, f8_narrow8<BF>(h[k]));
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(h[k][i], h[k][i], s);
      ss += s;
    }
  }
  ss = group_sum(ss, part);
  double exact = ss;
  const bool fits = ss < INFINITY;
  if (!fits) {  // (the same in every thread)
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (threadIdx.x + k * blockDim.x < (uint32_t)chunks)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += (double)h[k][i] * (double)h[k][i];
    exact = group_sum(s, part64);
  }
  const float rstd = 1.0f / sqrtf(ss / (float)a.n + a.eps);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
    const bool live = c < chunks;
    float u[8], g[8];
    if (a.gamma) f8_widen8<BF>(ldg(reinterpret_cast<const u32x4 *>(a.gamma) + min(c, chunks - 1)), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = a.gamma ? h[k][i] * g[i] : h[k][i];
    const uint32_t top = row16_umax(live ? magnitude8(u) : 0u);
    float post = rstd;
    if (!fits || !(top < kInfBits) || __builtin_bit_cast(float, top) < 1e-30f) {
      const double f = 1.0 / sqrt(exact / a.n + (double)a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = (float)((double)h[k][i] * f * (a.gamma ? (double)g[i] : 1.0));
      post = 1.f;
    }
    put_block<BF>(a.out, u, post, live, row, a.n, c);
  }
}

// e^-z 2^-less: e^-z = 2^t (1 + r ln 2) with t = -z log2 e rounded and r what that lost (so t is not to
// be formed anew, unrounded, where less is subtracted).
__device__ __forceinline__ float exp_neg(float z, float less) {
#pragma clang fp contract(off)
  constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f;  // log2 e - kLog2e
  const float t = -z * kLog2e;
  const float r = fmaf(-z, kLog2eRest, fmaf(-z, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t - less);
  return fmaf(e * 0.693147181f, r, e);
}

// 1 / (1 + e^-z) within about 2 ulp for z >= kLowGate, in ten instructions (the library's exponential
// and division take three times that, and bound the kernel: 46 us for 2048 x 17408).  The reciprocal
// gets one Newton step.
constexpr float kLowGate = -80.f;
constexpr uint32_t kLowBitsF16 = 0xD500, kLowBitsBf16 = 0xC2A0;  // its bits
__device__ __forceinline__ float sigmoid(float z) {
  const float d = 1.0f + exp_neg(fminf(fmaxf(z, kLowGate), 200.f), 0.f);  // (1 from there on; a NaN's result is multiplied by it)
  const float q = __builtin_amdgcn_rcpf(d);
  return fmaf(fmaf(-d, q, 1.0f), q, q);
}

// z / (1 + e^-z) u for z below kLowGate, where the sigmoid leaves f32's normal numbers, but not its
// product with a large u: 1 + e^-z is e^-z there, to 2^-115, and is formed without a factor of 2^144 that the
// product in 64 bits gets back.  From z = -187 on the result is below 2^-134, half of the smallest
// number that 16 bits hold, whatever u; it keeps its sign, and u = infinity stays one.
__device__ __forceinline__ float silu_mul_low(float z, float u) {
  const float d = exp_neg(fmaxf(z, -187.f), 144.f);
  float q = __builtin_amdgcn_rcpf(d);
  q = fmaf(fmaf(-d, q, 1.0f), q, q);
  const double f = z < -187.f ? (double)(z - z) - 0x1p-300 : (double)z * (double)q * 0x1p-144;  // (-infinity: NaN)
  return (float)(f * (double)u);
}

// The largest of eight 16-bit words as whole numbers.
__device__ __forceinline__ uint32_t top_u16(const u32x4 &w) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = __builtin_bit_cast(u16x2, w[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i]));
  return max((uint32_t)m[0], (uint32_t)m[1]);
}

// One chunk of eight channels a thread; the rows' blocks, each 16 threads, follow each other, two
// blocks of a thread under way.  2048 x 17408 (179 MB): 34 us, 5.3 TB/s; its sigmoids and conversions
// are about as long.  A wave that has a gate below kLowGate forms its blocks again (a choice between
// the two for each channel took 38 us); it reads them again, which leaves the registers as they are.
template <bool BF>
__global__ __launch_bounds__(256) void silu_mul_kernel(F8Act a, int blocks, uint32_t items) {
  for (uint32_t first = blockIdx.x * 32; first < items; first += gridDim.x * 32) {
    u32x4 gs[2], us[2];
    uint32_t row[2];
    int chunk[2];
    bool live[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t it = first + 16 * k + (threadIdx.x >> 4);
      row[k] = min(it, items - 1) / (uint32_t)blocks;
      chunk[k] = (int)(min(it, items - 1) - row[k] * blocks) * 16 + (threadIdx.x & 15);
      live[k] = it < items && chunk[k] * 8 < a.n;
      const uint16_t *p = a.x + (size_t)row[k] * a.x_row + 8 * (chunk[k] * 8 < a.n ? chunk[k] : 0);
      gs[k] = ldg(reinterpret_cast<const u32x4 *>(p));
      us[k] = ldg(reinterpret_cast<const u32x4 *>(p + a.n));
    }
    uint32_t far = 0;  // gates below kLowGate are above its bits
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float g[8], u[8];
      f8_widen8<BF>(gs[k], g);
      f8_widen8<BF>(us[k], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] *= g[i] * sigmoid(g[i]);
      put_block<BF>(a.out, u, 1.f, live[k], row[k], a.n, chunk[k]);
      far = max(far, top_u16(gs[k]));
    }
    if (__any(far > (BF ? kLowBitsBf16 : kLowBitsF16))) {  // (hardly ever)
#pragma clang loop unroll(disable)
      for (int k = 0; k < 2; ++k) {
        const uint32_t it = first + 16 * k + (threadIdx.x >> 4);
        const uint32_t r = min(it, items - 1) / (uint32_t)blocks;
        const int c = (int)(min(it, items - 1) - r * blocks) * 16 + (threadIdx.x & 15);
        const uint16_t *p = a.x + (size_t)r * a.x_row + 8 * (c * 8 < a.n ? c : 0);
        float g[8], u[8];
        f8_widen8<BF>(ldg(reinterpret_cast<const u32x4 *>(p)), g);
        f8_widen8<BF>(ldg(reinterpret_cast<const u32x4 *>(p + a.n)), u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[i] = g[i] < kLowGate ? silu_mul_low(g[i], u[i]) : u[i] * (g[i] * sigmoid(g[i]));
          asm volatile("" : "+v"(u[i]));  // (not all at once: registers)
        }
        put_block<BF>(a.out, u, 1.f, it < items && c * 8 < a.n, r, a.n, c);
      }
    }
  }
}

template <bool BF>
hipError_t norm(const F8Norm &a, hipStream_t stream) {
  const int chunks = a.n >> 3;
  const int threads = chunks >= 1024 ? 1024 : (chunks + 63) / 64 * 64;
  const int v = (chunks + threads - 1) / threads;
  if (v == 1) norm_kernel<BF, 1><<<a.rows, threads, 0, stream>>>(a);
  else if (v == 2) norm_kernel<BF, 2><<<a.rows, threads, 0, stream>>>(a);
  else norm_kernel<BF, 4><<<a.rows, threads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_norm(const F8Norm &a, hipStream_t stream) {
  return a.bf16 ? norm<true>(a, stream) : norm<false>(a, stream);
}

hipError_t launch_f8_silu_mul(const F8Act &a, hipStream_t stream) {
  const int blocks = (a.n + kF8Block - 1) / kF8Block;
  const uint32_t items = (uint32_t)a.rows * (uint32_t)blocks;
  const uint32_t grid = min((items + 31) / 32, 1u << 20);
  if (a.bf16) silu_mul_kernel<true><<<grid, 256, 0, stream>>>(a, blocks, items);
  else silu_mul_kernel<false><<<grid, 256, 0, stream>>>(a, blocks, items);
  return hipGetLastError();
}

}  // namespace trellis
