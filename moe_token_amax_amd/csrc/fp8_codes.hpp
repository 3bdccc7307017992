// E4M3 codes of blocks of 128 values held by 16 lanes, 8 values each.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "dpp_row.hpp"

namespace w8a8 {

// Scale of a block from the bits of its largest magnitude. alg 1: the smallest
// power of two (at least 2^-126) not below amax / 448. NaN stays NaN.
__device__ __forceinline__ float block_scale(uint32_t amax_bits, int alg) {
  const float s = __uint_as_float(amax_bits) / 448.0f;
  if (alg == 0 || !(s > 0.0f) || !(s <= 3.402823466e38f)) return s;
  return __uint_as_float((__float_as_uint(s) + 0x7FFFFFu) & 0xFF800000u);
}

// fl(x / s) clamped to +-448. With y = fl(1 / s) correctly rounded, q = fl(x y) and
// r = x - q s (exact in one fused operation), fl(q + r y) is the correctly rounded
// quotient (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): three operations instead of the division's
// eleven, the reciprocal shared by the block. Exact means no underflow: with s in
// [2^-80, 2^80] r is representable for every quotient above 2^-22, and a smaller
// one has code 0 anyway, whose sign is x's (x = -0 gives q + r y = +0). Other
// scales divide.
__device__ __forceinline__ float quotient(float x, float s, float y) {
  const float q = x * y;
  const float t = __builtin_fmaf(__builtin_fmaf(-q, s, x), y, q);
  return __builtin_amdgcn_fmed3f(__builtin_copysignf(t, x), -448.0f, 448.0f);
}

__device__ __forceinline__ uint2 pack_codes(const float (&t)[8]) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], hi, true);
  return uint2{(uint32_t)lo, (uint32_t)hi};
}

// Codes of this lane's 8 values of a block of 128 held by 16 lanes, and its scale.
__device__ __forceinline__ uint2 quant_block(const float (&v)[8], int alg, float& s) {
  uint32_t am = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) am = max(am, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  s = block_scale(row_max_u32(am), alg);
  float t[8];
  if (s >= 0x1p-80f && s <= 0x1p+80f) {
    const float y = 1.0f / s;
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = quotient(v[j], s, y);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      t[j] = s > 0.0f ? v[j] / s : 0.0f;  // s NaN: 0
      // an infinity over its infinite scale stays NaN (the limits alone would make it -448)
      if (!__builtin_isnan(t[j])) t[j] = fminf(fmaxf(t[j], -448.0f), 448.0f);
    }
  }
  return pack_codes(t);
}

}  // namespace w8a8
