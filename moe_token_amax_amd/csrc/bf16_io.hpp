// BF16 rows in registers: accesses of 8 values at any address, conversions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace w8a8 {

// 16 and 8 bytes at any BF16 address: gfx950 loads and stores them in one
// instruction, at full rate where they happen to be aligned, so odd widths need no
// path of their own (in single values the quantizer took 20.3 us for 4096 x 4097,
// now 10.1, and a product's outputs 52 us for 5366 x 4089 x 197, now 34)
struct __attribute__((packed, aligned(2))) Bytes16 {
  uint32_t w[4];
};
struct __attribute__((packed, aligned(2))) Bytes8 {
  uint32_t w[2];
};

// fp32 -> BF16 with the hardware conversion: half to even, NaN stays NaN
__device__ __forceinline__ uint16_t to_bf16(float f) {
  const __bf16 b = (__bf16)f;
  return __builtin_bit_cast(uint16_t, b);
}

// 8 values from src, n of them in the row (0 past it), and with PAIR 8 more from
// src + next (under one branch, so that both loads are in flight together)
template <bool PAIR>
__device__ __forceinline__ void load8(const uint16_t* src, int64_t next, int64_t n, float (&v)[8], float (&u)[8]) {
  Bytes16 a{}, b{};
  if (n >= 8) {
    a = *reinterpret_cast<const Bytes16*>(src);
    if (PAIR) b = *reinterpret_cast<const Bytes16*>(src + next);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < n) {
        a.w[j / 2] |= (uint32_t)src[j] << (16 * (j & 1));
        if (PAIR) b.w[j / 2] |= (uint32_t)src[next + j] << (16 * (j & 1));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(a.w[j] << 16);
    v[2 * j + 1] = __uint_as_float(a.w[j] & 0xFFFF0000u);
    if (PAIR) {
      u[2 * j] = __uint_as_float(b.w[j] << 16);
      u[2 * j + 1] = __uint_as_float(b.w[j] & 0xFFFF0000u);
    }
  }
}

}  // namespace w8a8
