// Device-side building blocks of the 4-bit key/value cache (format: include/trellis_kv4.h).
#pragma once
#include "launch.h"
#include "launch_kv4.h"
#include "trellis_device.h"

namespace trellis {

constexpr float kRsqrt128 = 0.08838834764831845f;

// Error-word bits (TRELLIS_KV4_ERR_*).
__device__ __forceinline__ void kv4_error(uint32_t *errword, uint32_t bit) {
  __hip_atomic_fetch_or(errword, bit, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// 16-bit element types.  bf16 is rounded to nearest even; a NaN stays one.
template <bool BF>
__device__ __forceinline__ float kv4_widen(uint16_t v) {
  return BF ? __builtin_bit_cast(float, (uint32_t)v << 16) : h2f(v);
}
template <bool BF>
__device__ __forceinline__ uint16_t kv4_narrow(float f) {
  if (!BF) return f2h(f);
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

// log2 of a page's tokens (16 .. 256): positions are split by shift and mask.
__device__ __forceinline__ int kv4_page_log2(int page_size) { return __builtin_ctz(page_size); }

// Where one (page, head) chunk's parts lie, in bytes from its start: T tokens, NB blocks.
struct Kv4Chunk {
  int T, NB;
  __device__ __forceinline__ int k_code(int nb, int t) const { return (nb * T + t) * 64; }
  __device__ __forceinline__ int v_code(int nb, int t) const { return ((NB + nb) * T + t) * 64; }
  __device__ __forceinline__ int k_scale(int nb, int t) const { return 128 * NB * T + (nb * T + t) * 2; }
  __device__ __forceinline__ int v_scale(int nb, int t) const { return 128 * NB * T + ((NB + nb) * T + t) * 2; }
  __device__ __forceinline__ int bytes() const { return 132 * NB * T; }
};

// The chunk of (layer, page, head); 64-bit, a pool may be far over 4 GiB.
__device__ __forceinline__ char *kv4_chunk(const trellis_kv4_cache &c, int layer, int page, int head) {
  const size_t chunk = (size_t)132 * (c.head_dim >> 7) * c.page_size;
  return static_cast<char *>(c.pool) + (((size_t)layer * c.n_pages + page) * c.n_kv_heads + head) * chunk;
}

// The sequence of a row: how many of cu[1..n_seq] are <= row.  The 16 lanes of a DPP row share
// the count (lane i takes every 16th entry), so the loads are in flight together.
__device__ __forceinline__ int kv4_seq_of(const int32_t *cu, int n_seq, int row, int lane16) {
  int n = 0;
  for (int j = lane16; j < n_seq; j += 16) n += ldg(cu + j + 1) <= row;
  n += __builtin_amdgcn_update_dpp(0, n, 0xB1, 0xF, 0xF, true);
  n += __builtin_amdgcn_update_dpp(0, n, 0x4E, 0xF, 0xF, true);
  n += __builtin_amdgcn_update_dpp(0, n, 0x141, 0xF, 0xF, true);  // the other four of eight
  n += __builtin_amdgcn_update_dpp(0, n, 0x128, 0xF, 0xF, true);
  return n;
}

// A row's place: its page and place in it, or page = -1 where cu, the slot, the length or the
// table does not give one (nothing of the table is read at an index out of its bounds).
struct Kv4Place {
  int page, at;
};
__device__ __forceinline__ Kv4Place kv4_place(const trellis_kv4_cache &c, const trellis_kv4_batch &b, int row,
                                              int lane16) {
  Kv4Place r{-1, 0};
  const int s = kv4_seq_of(b.cu, b.n_seq, row, lane16);
  if (s >= b.n_seq) return r;
  const int slot = b.slots ? ldg(b.slots + s) : s;
  if ((uint32_t)slot >= (uint32_t)b.n_slots) return r;
  const int c0 = ldg(b.cu + s), c1 = ldg(b.cu + s + 1);
  const long long pos = (long long)ldg(b.lens + slot) - c1 + row;  // len - (c1 - c0) + (row - c0)
  if (row < c0 || pos < 0 || pos >= (long long)b.max_pages * c.page_size) return r;
  const int page = ldg(b.table + (size_t)slot * b.max_pages + ((int)pos >> kv4_page_log2(c.page_size)));
  if ((uint32_t)page >= (uint32_t)c.n_pages) return r;
  r.page = page;
  r.at = (int)pos & (c.page_size - 1);
  return r;
}

// Kind n of a row's 2 * n_kv_heads * NB blocks: keys' blocks head by head, then the values'.
struct Kv4Kind {
  int head, nb;
  bool is_v;
};
__device__ __forceinline__ Kv4Kind kv4_kind(const trellis_kv4_cache &c, int n) {
  const int log_nb = c.head_dim >> 8, half = c.n_kv_heads << log_nb;
  const bool is_v = n >= half;
  const int k = is_v ? n - half : n;
  return {k >> log_nb, k & log_nb, is_v};
}

// H_128 (unnormalised) over 16 lanes holding elements 8i .. 8i+7, strides 1, 2, 4 .. 64, up to a
// sign a lane and the order of the lanes, in one instruction an element and stage across lanes:
// v + c v', with v' the partner's and c = -1 in a pair's second lane, is the
// butterfly with that lane's result negated, and all of a later stage's partners carry the same
// negations.  The third stage pairs i with 7 - i, which one lane pattern reaches and i ^ 4 does
// not; H_8 over the masks 1, 2, 7 is H_8 over 1, 2, 4 with its outputs in another order.  Lane i
// ends with elements 8 k .. 8 k + 7, k = kv4_fwht16_place(i), times kv4_fwht16_sign(i).
__device__ __forceinline__ int kv4_fwht16_place(int i) {
  const int b2 = (i >> 2) & 1, k0 = (i & 1) ^ b2, k1 = ((i >> 1) & 1) ^ b2;
  return (i & 8) | ((k0 ^ k1 ^ b2) << 2) | (k1 << 1) | k0;
}
__device__ __forceinline__ float kv4_fwht16_sign(int i) { return (__builtin_popcount(i & 15) & 1) ? -1.f : 1.f; }
__device__ __forceinline__ void kv4_fwht16_signed(float (&v)[8], int i) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if ((t & h) == 0) {
        const float a = v[t], b = v[t + h];
        v[t] = a + b;
        v[t + h] = a - b;
      }
  const int b2 = (i >> 2) & 1;
  const float c1 = ((i & 1) ^ b2) ? -1.f : 1.f, c2 = (((i >> 1) & 1) ^ b2) ? -1.f : 1.f;
  const float c7 = b2 ? -1.f : 1.f, c8 = (i & 8) ? -1.f : 1.f;
  // One block: a lane pattern's operand must have been written at least two instructions before
  // (the leading wait; then every element is eight instructions old).
  asm("s_nop 4\n\t"
#define KV4_STAGE(c, pattern)                                                                                          \
  "v_fmac_f32_dpp %0, %0, " c " " pattern "\n\tv_fmac_f32_dpp %1, %1, " c " " pattern                                  \
  "\n\tv_fmac_f32_dpp %2, %2, " c " " pattern "\n\tv_fmac_f32_dpp %3, %3, " c " " pattern                            \
  "\n\tv_fmac_f32_dpp %4, %4, " c " " pattern "\n\tv_fmac_f32_dpp %5, %5, " c " " pattern                            \
  "\n\tv_fmac_f32_dpp %6, %6, " c " " pattern "\n\tv_fmac_f32_dpp %7, %7, " c " " pattern "\n\t"
      KV4_STAGE("%8", "quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf bound_ctrl:1")
      KV4_STAGE("%9", "quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf bound_ctrl:1")
      KV4_STAGE("%10", "row_half_mirror row_mask:0xf bank_mask:0xf bound_ctrl:1")
      KV4_STAGE("%11", "row_ror:8 row_mask:0xf bank_mask:0xf bound_ctrl:1")
#undef KV4_STAGE
      : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7])
      : "v"(c1), "v"(c2), "v"(c7), "v"(c8));
}

// The largest of 16 lanes' numbers.
__device__ __forceinline__ uint32_t kv4_max16(uint32_t v) {
  const auto up = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  v = up(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true));
  v = up(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true));
  v = up(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true));
  return up(v, __builtin_amdgcn_update_dpp(0, v, 0x128, 0xF, 0xF, true));
}

template <bool BF>
__device__ __forceinline__ void kv4_unpack8(u32x4 p, float (&v)[8]) {
#pragma unroll
  for (int t = 0; t < 8; ++t) v[t] = kv4_widen<BF>((t & 1) ? (uint16_t)(p[t >> 1] >> 16) : (uint16_t)p[t >> 1]);
}

template <bool BF>
__device__ __forceinline__ u32x4 kv4_pack8(const float (&v)[8]) {
  u32x4 o;
#pragma unroll
  for (int t = 0; t < 4; ++t) o[t] = (uint32_t)kv4_narrow<BF>(v[2 * t]) | ((uint32_t)kv4_narrow<BF>(v[2 * t + 1]) << 16);
  return o;
}

// Eight E2M1 codes (one word, element 0 in the low nibble) as numbers.
__device__ __forceinline__ void kv4_values8(uint32_t w, float (&v)[8]) {
  const floatx2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const floatx2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const floatx2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const floatx2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
}

}  // namespace trellis
