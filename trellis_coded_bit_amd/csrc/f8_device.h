// Device-side building blocks of the block-scaled FP8 operators (format: include/trellis_f8.h).
#pragma once
#include "launch.h"
#include "launch_f8.h"
#include "trellis_device.h"

namespace trellis {

// Bytes of an array from which on a kernel that passes over it once leaves the caches alone (all
// L2 caches together hold 32 MB).  Rows gathered and combined for 4097 tokens: 117 us so, 140 without;
// the gradients for 4096: 214 and 233.  On either side of the bound, us through the caches | past them: rows
// gathered 6.6 | 5.8 (16 MB), 9.3 | 7.6 (24 MB), 11.3 | 10.0 (32 MB), combined 5.9 | 5.7, 7.7 | 6.9, 9.3 | 8.2,
// one after the other 12.0 | 11.3, 16.0 | 14.3, 18.9 | 17.9.  Past them is no slower below the bound
// either; there the rows are left in the caches for a product that reads them next, which these leave out.
constexpr size_t kF8Once = (size_t)24 << 20;

// 16-bit element types.  bf16 is rounded to nearest even; a NaN stays one.
template <bool BF>
__device__ __forceinline__ float f8_widen(uint16_t v) {
  return BF ? __builtin_bit_cast(float, (uint32_t)v << 16) : h2f(v);
}
template <bool BF>
__device__ __forceinline__ uint16_t f8_narrow(float f) {
  if (!BF) return f2h(f);
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

// Eight 16-bit elements of a 16-byte word.
template <bool BF>
__device__ __forceinline__ void f8_widen8(const u32x4 &w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = f8_widen<BF>((uint16_t)(w[i] & 0xFFFFu));
    v[2 * i + 1] = f8_widen<BF>((uint16_t)(w[i] >> 16));
  }
}
template <bool BF>
__device__ __forceinline__ u32x4 f8_narrow8(const float (&v)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (uint32_t)f8_narrow<BF>(v[2 * i]) | ((uint32_t)f8_narrow<BF>(v[2 * i + 1]) << 16);
  return w;
}

// Stores through the global address space (see ldg).
template <typename T>
__device__ __forceinline__ void stg(T *p, const T &v) {
  *(__attribute__((address_space(1))) T *)p = v;
}

// The same for what is read or written once and is more than the caches keep (NT): it leaves them to
// what is used again.
template <bool NT, typename T>
__device__ __forceinline__ T ldg_once(const T *p) {
  return NT ? __builtin_nontemporal_load((const __attribute__((address_space(1))) T *)p) : ldg(p);
}
template <bool NT, typename T>
__device__ __forceinline__ void stg_once(T *p, const T &v) {
  if (NT) __builtin_nontemporal_store(v, (__attribute__((address_space(1))) T *)p);
  else stg(p, v);
}

// The largest magnitude, as bits without sign (a NaN's are above an infinity's, which are above
// every number's), over the 16 lanes of a DPP row.
__device__ __forceinline__ uint32_t row16_umax(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xF, 0xF, true));
  return m;
}
__device__ __forceinline__ uint32_t magnitude8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
  return m;
}

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr float kF8Max = 448.0f, kMinNormal = 1.17549435e-38f;

// A block's scale and the factor that turns its values into codes' values, from the largest
// magnitude (bits) of values that `post` multiplies.  The codes do not depend on post, so its
// rounding does not reach them: only 448 / a and the product with it are rounded before E4M3 is.
struct F8Scale {
  float scale, inv;
};
__device__ __forceinline__ F8Scale f8_scale(uint32_t top, float post) {
  const float a = __builtin_bit_cast(float, top);
  F8Scale r;
  r.scale = a * post / kF8Max;
  r.inv = kF8Max / a;
  if (!(top < kInfBits) || !(r.scale < INFINITY)) r = {NAN, 0.f};
  else if (r.scale < kMinNormal) r = {0.f, 0.f};
  return r;
}
// Codes of eight values; inv = 0 gives zeros also for what is not a number.
__device__ __forceinline__ u32x2 f8_codes(const float (&v)[8], float inv) {
  u32x2 w = {0, 0};
  if (inv != 0.f) {
    float c[8];
    // (a * (448 / a) may round to just above 448, which would still round to 448; the clamp keeps
    // the conversion away from its saturation)
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(v[i] * inv, -kF8Max), kF8Max);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i], c[4 * i + 1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i + 2], c[4 * i + 3], p, true);
    }
  }
  return w;
}

__device__ __forceinline__ void f8_error(uint32_t *errword) {
  __hip_atomic_fetch_or(errword, kErrBadEntry, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace trellis
