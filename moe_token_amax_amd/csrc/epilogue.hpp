// Activations of the fused epilogues, on fp32 sums.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/w8a8.h"
#include "bf16_io.hpp"
#include "device_common.hpp"

namespace w8a8 {

// v / (1 + e^-t) by the hardware's exponential and reciprocal (1 ulp each; the
// exponent's rounding makes it a few 2^-24 |t| more, far inside a BF16 step). Ends:
// below t = -87 the reciprocal, which knows no subnormals, and then e^-t = inf give v * 0
// for a value under 2^-118 (BF16 would hold it; scaling the exponential would cost every
// output another reciprocal); NaN stays NaN.
__device__ __forceinline__ float times_sigmoid(float v, float t) {
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t * -1.44269504f));
}

// v Phi(v): erfc by M. Abramowitz and I. Stegun, Handbook of Mathematical Functions,
// 7.1.26 (within 1.5e-7; of erfc itself 0.05 % at v = -4, 0.4 % at -6, 2 % at -10), times
// e^(-v^2 / 2)
__device__ __forceinline__ float gelu_erf(float v) {
  const float z = fabsf(v) * 0.70710678f;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, z, 1.0f));
  float s = 1.061405429f;
  s = __builtin_fmaf(s, t, -1.453152027f);
  s = __builtin_fmaf(s, t, 1.421413741f);
  s = __builtin_fmaf(s, t, -0.284496736f);
  s = __builtin_fmaf(s, t, 0.254829592f);
  const float tail = 0.5f * s * t * __builtin_amdgcn_exp2f(z * z * -1.44269504f);  // Phi(-|v|)
  return v * (v < 0.0f ? tail : 1.0f - tail);
}

__device__ __forceinline__ float activate(int act, float v) {
  switch (act) {  // the same in every lane
    case W8A8_ACT_RELU: return v < 0.0f ? 0.0f : v;
    case W8A8_ACT_SILU: return times_sigmoid(v, v);
    case W8A8_ACT_GELU: return gelu_erf(v);
    // 0.5 (1 + tanh u) = 1 / (1 + e^(-2u)), u = sqrt(2 / pi) (v + 0.044715 v^3)
    case W8A8_ACT_GELU_TANH: return times_sigmoid(v, v * __builtin_fmaf(0.0713548163f, v * v, 1.59576912f));
    default: return v;
  }
}

// four values behind one choice
__device__ __forceinline__ void activate4(int act, float (&v)[4]) {
#define W8A8_EACH(expr)                            \
  {                                                \
    _Pragma("unroll") for (int t = 0; t < 4; ++t) { \
      const float x = v[t];                        \
      v[t] = expr;                                 \
    }                                              \
    break;                                         \
  }
  switch (act) {
    case W8A8_ACT_RELU: W8A8_EACH(activate(W8A8_ACT_RELU, x))
    case W8A8_ACT_SILU: W8A8_EACH(activate(W8A8_ACT_SILU, x))
    case W8A8_ACT_GELU: W8A8_EACH(activate(W8A8_ACT_GELU, x))
    case W8A8_ACT_GELU_TANH: W8A8_EACH(activate(W8A8_ACT_GELU_TANH, x))
    default: break;
  }
#undef W8A8_EACH
}

constexpr int kAnyAct = -1;

// run(ACT) for act, so that a loop over rows holds no choice of it (some ten branches an
// output: 0.7 us for every 16 rows of a tile)
template <bool SWIGLU, class Run>
__device__ __forceinline__ void for_act(int act, Run run) {
  switch (act) {  // the same in every lane
    case W8A8_ACT_SWIGLU:
      if constexpr (SWIGLU) run(std::integral_constant<int, W8A8_ACT_SWIGLU>{});
      break;
    case W8A8_ACT_RELU: run(std::integral_constant<int, W8A8_ACT_RELU>{}); break;
    case W8A8_ACT_SILU: run(std::integral_constant<int, W8A8_ACT_SILU>{}); break;
    case W8A8_ACT_GELU: run(std::integral_constant<int, W8A8_ACT_GELU>{}); break;
    case W8A8_ACT_GELU_TANH: run(std::integral_constant<int, W8A8_ACT_GELU_TANH>{}); break;
    default: run(std::integral_constant<int, W8A8_ACT_NONE>{}); break;
  }
}

// What is added where there is no bias or no residual, -0 (v + -0 is v, also where v is
// -0): a pair of it in BF16.
constexpr uint32_t kNothing2 = 0x80008000u;

__device__ __forceinline__ float bf16_of(const Bytes8& u, int t) {
  return __uint_as_float(t & 1 ? u.w[t >> 1] & 0xFFFF0000u : u.w[t >> 1] << 16);
}

// n of four BF16 values as they lie in memory, -0 past them. WHOLE: n is 4.
template <bool WHOLE>
__device__ __forceinline__ Bytes8 load_raw4(const uint16_t* src, int n) {
  if (WHOLE) return *reinterpret_cast<const Bytes8*>(src);
  uint32_t u[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) u[t] = t < n ? src[t] : kNothing2 & 0xFFFFu;
  return Bytes8{{u[0] | (u[1] << 16), u[2] | (u[3] << 16)}};
}

// up to 4 neighbouring BF16 values (0 past n of them)
__device__ __forceinline__ void load_bf16x4(const uint16_t* src, int n, float (&v)[4]) {
  if (n >= 4) {
    const Bytes8 u = *reinterpret_cast<const Bytes8*>(src);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      v[2 * t] = __uint_as_float(u.w[t] << 16);
      v[2 * t + 1] = __uint_as_float(u.w[t] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = t < n ? bf16_to_f32(src[t]) : 0.0f;
  }
}

}  // namespace w8a8
