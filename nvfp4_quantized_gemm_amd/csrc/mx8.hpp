// MXFP8 encoding shared by the kernels that write it (gfx950): 32-value blocks along K, one E8M0
// scale byte b (X = 2^(b - 127)) and one E4M3 code per value.
//
// Definition (the OCP microscaling rule, as for MXFP4): with E the fp32 exponent field of the
// block's largest magnitude, b = max(E - 8, 0), i.e. X = 2^(floor(log2 amax) - 8) and 8 the largest
// E4M3 exponent; the code is the E4M3 value nearest to v / X, ties to even, saturating at 448.
// v * 2^(127 - b) is exact (a power of two; the result is below 512), so the hardware's
// round-to-nearest-even conversion of it, clamped to 448 first (unclamped it gives NaN above 464),
// is the code.  A block that holds an infinity or a NaN gets b = 255 (the E8M0 NaN) and NaN codes, so that
// neither a dequantization nor a product turns it into numbers.
#pragma once
#include "common.hpp"

namespace nvfp4 {

constexpr int kMx8Blk = 32;
constexpr float kMx8Max = 448.0f;

__device__ __forceinline__ uint32_t swap_lane1(uint32_t v) { return __float_as_uint(swap_lane1(__uint_as_float(v))); }
__device__ __forceinline__ uint32_t swap_lane2(uint32_t v) { return __float_as_uint(swap_lane2(__uint_as_float(v))); }

// Largest magnitude (as its bits, so that a NaN counts as the largest) of a block whose 32 values
// lie in 4 adjacent lanes, 8 each.
__device__ __forceinline__ uint32_t mx8_amax_bits(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = max(m, swap_lane1(m));
  return max(m, swap_lane2(m));
}
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t amax_bits) {
  const uint32_t E = amax_bits >> 23;
  return E == 255u ? 255u : (E > 8u ? E - 8u : 0u);
}
// 2^(127 - b) for the finite bytes the rule gives (b <= 246)
__device__ __forceinline__ float mx8_inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }
// X = 2^(b - 127); NaN for b = 255
__device__ __forceinline__ float mx8_scale_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fc00000u : (b ? b << 23 : 0x00400000u));
}

__device__ __forceinline__ uint32_t mx8_encode4(float a, float b, float c, float d) {
  a = fminf(fmaxf(a, -kMx8Max), kMx8Max);
  b = fminf(fmaxf(b, -kMx8Max), kMx8Max);
  c = fminf(fmaxf(c, -kMx8Max), kMx8Max);
  d = fminf(fmaxf(d, -kMx8Max), kMx8Max);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
// The 8 codes of a lane's values under scale byte b.
__device__ __forceinline__ u32x2 mx8_encode8(const float (&v)[8], uint32_t b) {
  if (b == 255u) return u32x2{0x7f7f7f7fu, 0x7f7f7f7fu};
  const float m = mx8_inv_scale(b);
  return u32x2{mx8_encode4(v[0] * m, v[1] * m, v[2] * m, v[3] * m), mx8_encode4(v[4] * m, v[5] * m, v[6] * m, v[7] * m)};
}
__device__ __forceinline__ void mx8_decode8(const u32x2 &c, uint32_t b, float (&v)[8]) {
  const float X = mx8_scale_value(b);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
    v[4 * i] = lo.x * X;
    v[4 * i + 1] = lo.y * X;
    v[4 * i + 2] = hi.x * X;
    v[4 * i + 3] = hi.y * X;
  }
}

// Eight consecutive elements of one lane, fp32 or bf16 (DT 0 / 1): 32 or 16 bytes.
template <int DT>
struct Vec8 {
  static constexpr int kWords = DT == 0 ? 2 : 1;
  u32x4 w[kWords];
  template <bool NT>
  __device__ __forceinline__ void load(const void *base, int64_t elem) {
    const uint8_t *p = static_cast<const uint8_t *>(base) + elem * (DT == 0 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = load16<NT>(p + 16 * i);
  }
  template <bool NT>
  __device__ __forceinline__ void store(void *base, int64_t elem) const {
    uint8_t *p = static_cast<uint8_t *>(base) + elem * (DT == 0 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < kWords; ++i) store16<NT>(p + 16 * i, w[i]);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (DT == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i / 4][i % 4]);
    } else {
      SegIn<1>::unpack(w[0], v);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    if constexpr (DT == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i / 4][i % 4] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x2 h = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
        w[0][i] = __builtin_bit_cast(uint32_t, h);
      }
    }
  }
};

}  // namespace nvfp4
