// Internal launcher of the RMS norm kernels (host side). Arguments are checked by
// the C ABI layer before it is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8a8 {

enum NormFormat { kNormBf16 = 0, kNormInt8 = 1, kNormFp8b = 2, kNormMx = 3 };

struct NormArgs {
  const uint16_t* x;         // BF16 [M, K], row stride ldx
  int64_t ldx;
  const uint16_t* residual;  // BF16 [M, K], row stride ldr, or null
  int64_t ldr;
  uint16_t* h;               // x + residual, row stride ldh (may be the residual itself); null without a residual
  int64_t ldh;
  const uint16_t* weight;    // BF16 [K] or null (1)
  double eps;
  int64_t M, K;
  uint16_t* y;               // BF16 [M, K], row stride ldy, or null
  int64_t ldy;
  uint8_t* q;                // codes, row stride ldq (kNormBf16: unused)
  int64_t ldq;
  void* scale;               // float [M]; float [ceil(K/128)][M]; uint8 [M][K/32]
  int scale_alg;
};
hipError_t launch_rms_norm(int format, const NormArgs& p, hipStream_t stream);

}  // namespace w8a8
