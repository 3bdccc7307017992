// RMS norm of BF16 rows for gfx950, the residual added first, the result in 8 bits
// with scales as the quantized products take it, and in BF16 where asked:
//
//   h = BF16(x + residual), r = fl32(1 / sqrt(sum h^2 / K + eps)), n = fl32(fl32(h r) w)
//   INT8 per row: s = fl32(max|n| / 127), code = rint(fl32(n / s))
//   E4M3 per 128 columns, MX E4M3 per 32: the rules of the two quantizers on n
//
// n is quantized as the fp32 number it is, with no BF16 between, and h is the BF16 that
// the stream keeps, so that the norm of what was stored is what was quantized. The sum
// runs in doubles: a square of a BF16 value is exact there, and the sum so nearly that
// r, and with it every code, does not depend on the order of the additions (two orders
// differ by 1e-16, and change the float r with probability 1e-9 a row).
#include <algorithm>

#include "bf16_io.hpp"
#include "device_common.hpp"
#include "fp8_codes.hpp"
#include "launch.hpp"
#include "norm.hpp"

namespace w8a8 {

// 8 codes at any address
struct __attribute__((packed, aligned(1))) Codes8 {
  uint32_t w[2];
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// 8 values from src, n of them in the row (0 past it)
__device__ __forceinline__ Bytes16 load_row8(const uint16_t* src, int64_t n) {
  Bytes16 a{};
  if (n >= 8) {
    a = *reinterpret_cast<const Bytes16*>(src);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) a.w[j / 2] |= (uint32_t)src[j] << (16 * (j & 1));
  }
  return a;
}

__device__ __forceinline__ void store_row8(uint16_t* dst, int64_t n, const Bytes16& a) {
  if (n >= 8) {
    *reinterpret_cast<Bytes16*>(dst) = a;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) dst[j] = (uint16_t)(a.w[j / 2] >> (16 * (j & 1)));
  }
}

__device__ __forceinline__ float value_of(const Bytes16& a, int j) {
  return __uint_as_float(j & 1 ? a.w[j / 2] & 0xFFFF0000u : a.w[j / 2] << 16);
}

__device__ __forceinline__ Bytes16 to_bytes(const float (&v)[8]) {
  Bytes16 a;
#pragma unroll
  for (int j = 0; j < 4; ++j) a.w[j] = to_bf16(v[2 * j]) | ((uint32_t)to_bf16(v[2 * j + 1]) << 16);
  return a;
}

// Codes of this lane's 8 values of a group of 32 held by 4 lanes, and its E8M0 byte. A
// maximum that is not finite makes the byte NaN's (255) and the codes NaN.
__device__ __forceinline__ uint2 quant_mx(const float (&v)[8], int alg, uint8_t& byte) {
  uint32_t am = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) am = max(am, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0xB1, 0xF, 0xF, false));
  am = max(am, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)am, 0x4E, 0xF, 0xF, false));
  if (am >= 0x7F800000u) {
    byte = 255;
    return uint2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
  }
  const float amax = __uint_as_float(am);
  int e = -127;
  if (am) {
    e = __builtin_amdgcn_frexp_expf(amax) - 1 - 8;
    if (alg == 1 && __builtin_ldexpf(amax, -e) > 448.0f) ++e;
    e = max(e, -127);
  }
  byte = (uint8_t)(e + 127);
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = __builtin_amdgcn_fmed3f(__builtin_ldexpf(v[j], -e), -448.0f, 448.0f);
  return pack_codes(t);
}

__device__ __forceinline__ float norm_factor(const NormArgs& p, double sum) {
  return (float)(1.0 / __builtin_sqrt(sum / (double)p.K + p.eps));
}

__device__ __forceinline__ Bytes16 load_weight(const NormArgs& p, int64_t k0) {
  if (p.weight) return load_row8(p.weight + k0, p.K - k0);
  return Bytes16{{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}};
}

__device__ __forceinline__ Bytes16 add8(const Bytes16& x, const Bytes16& a) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = value_of(x, j) + value_of(a, j);
  return to_bytes(v);
}

// chunk c of x + residual, which goes to h
__device__ __forceinline__ Bytes16 load_sum(const NormArgs& p, int64_t row, int c) {
  const int64_t k0 = (int64_t)c * 8, n = p.K - k0;
  Bytes16 h = load_row8(p.x + row * p.ldx + k0, n);
  if (p.residual) {
    h = add8(h, load_row8(p.residual + row * p.ldr + k0, n));
    store_row8(p.h + row * p.ldh + k0, n, h);
  }
  return h;
}

// bits of max|n| of a chunk with `left` values
__device__ __forceinline__ uint32_t chunk_max(const Bytes16& h, const Bytes16& g, float r, int64_t left) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) top = max(top, __float_as_uint(value_of(h, j) * r * value_of(g, j)) & 0x7FFFFFFFu);
  return top;
}

// n of chunk c, quantized and (y) in BF16. s: the row's scale (INT8). Every lane of a
// block's 16 (4) takes part.
template <int FMT>
__device__ __forceinline__ void write_chunk(const NormArgs& p, int64_t row, int c, const Bytes16& h, const Bytes16& g,
                                            float r, float s) {
  const int64_t K = p.K, k0 = (int64_t)c * 8;
  float n[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) n[j] = k0 + j < K ? value_of(h, j) * r * value_of(g, j) : 0.0f;
  if (p.y) store_row8(p.y + row * p.ldy + k0, K - k0, to_bytes(n));
  if (FMT == kNormInt8) {
    const uint2 o = quant8(n, s);
    uint8_t* q = p.q + row * p.ldq + k0;
    if (k0 + 8 <= K) {
      *reinterpret_cast<Codes8*>(q) = Codes8{{o.x, o.y}};
    } else {
      for (int j = 0; k0 + j < K; ++j) q[j] = (uint8_t)((j < 4 ? o.x : o.y) >> (8 * (j & 3)));
    }
  } else if (FMT == kNormFp8b) {
    float bs;
    const uint2 o = quant_block(n, p.scale_alg, bs);
    *reinterpret_cast<uint2*>(p.q + row * p.ldq + k0) = o;
    if ((c & 15) == 0) reinterpret_cast<float*>(p.scale)[(int64_t)(c >> 4) * p.M + row] = bs;
  } else if (FMT == kNormMx) {
    uint8_t byte;
    const uint2 o = quant_mx(n, p.scale_alg, byte);
    *reinterpret_cast<uint2*>(p.q + row * p.ldq + k0) = o;
    if ((c & 3) == 0) reinterpret_cast<uint8_t*>(p.scale)[row * (K / 32) + (c >> 2)] = byte;
  }
}

// WPR wavefronts a row, CPL chunks of 8 values a lane: the row stays in registers
// between the sum, the maximum and the codes, and is read once. A workgroup walks over
// its rows and keeps the weight of its columns. HBM-bound: 8192 x 7168 with residual to
// INT8 97 us (411 MB, 4.25 TB/s; a copy 5.3), to E4M3 87, MX 84, BF16 alone 92 (470 MB); one
// row 4.7 (a sum and a maximum over 16 wavefronts, one behind the other, and a launch), MX
// 4.2, BF16 3.7. Odd addresses double the L1's look-ups, not the time (1237 x 4096 to E4M3
// and BF16 13.2, with rows 4097 apart 13.7).
template <int FMT, int CPL, int WPR>
__global__ __launch_bounds__(WPR >= 4 ? WPR * kWave : 256) void rms_norm_kernel(NormArgs p) {
  constexpr int kThreadsRow = WPR * kWave, kRows = WPR >= 4 ? 1 : 4 / WPR;
  __shared__ double sums[2][WPR];
  __shared__ uint32_t tops[2][WPR];
  const int t = threadIdx.x % kThreadsRow, lane = threadIdx.x & 63, wave = t / kWave;
  const int64_t K = p.K, KB = (K + 127) / 128;
  // chunks of a row; block-scaled rows are padded to whole blocks
  const int nchunk = (int)(FMT == kNormFp8b ? KB * 16 : (K + 7) / 8);
  Bytes16 g[CPL];
#pragma unroll
  for (int i = 0; i < CPL; ++i) g[i] = load_weight(p, (int64_t)(t + i * kThreadsRow) * 8);
  int par = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kThreadsRow; row < p.M;
       row += (int64_t)gridDim.x * kRows, par ^= 1) {
    const uint16_t* xr = p.x + row * p.ldx;
    Bytes16 h[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int64_t k0 = (int64_t)(t + i * kThreadsRow) * 8;
      h[i] = load_row8(xr + k0, K - k0);
    }
    if (p.residual) {
      const uint16_t* rr = p.residual + row * p.ldr;
      Bytes16 a[CPL];
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        const int64_t k0 = (int64_t)(t + i * kThreadsRow) * 8;
        a[i] = load_row8(rr + k0, K - k0);
      }
      uint16_t* hr = p.h + row * p.ldh;
#pragma unroll
      for (int i = 0; i < CPL; ++i) {
        const int64_t k0 = (int64_t)(t + i * kThreadsRow) * 8;
        h[i] = add8(h[i], a[i]);
        store_row8(hr + k0, K - k0, h[i]);
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double v = (double)value_of(h[i], j);
        sum = __builtin_fma(v, v, sum);
      }
    sum = wave_sum(sum);
    if (WPR > 1) {
      if (lane == 0) sums[par][wave] = sum;
      __syncthreads();
      sum = sums[par][0];
#pragma unroll
      for (int w = 1; w < WPR; ++w) sum += sums[par][w];
    }
    const float r = norm_factor(p, sum);
    float s = 0.0f;
    if (FMT == kNormInt8) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < CPL; ++i) top = max(top, chunk_max(h[i], g[i], r, K - (int64_t)(t + i * kThreadsRow) * 8));
      top = wave_max_u32(top);
      if (WPR > 1) {
        if (lane == 0) tops[par][wave] = top;
        __syncthreads();
        top = tops[par][0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) top = max(top, tops[par][w]);
      }
      s = __uint_as_float(top) / 127.0f;
      if (t == 0) reinterpret_cast<float*>(p.scale)[row] = s;
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = t + i * kThreadsRow;
      if (c < nchunk) write_chunk<FMT>(p, row, c, h[i], g[i], r, s);
    }
  }
}

// Rows past what registers hold: a 1024-thread workgroup a row, which goes through it
// once for the sum, once for the maximum (INT8) and once for the codes. A thread reads
// back the h that it wrote itself.
template <int FMT>
__global__ __launch_bounds__(1024) void rms_norm_long_kernel(NormArgs p) {
  __shared__ double sums[16];
  __shared__ uint32_t tops[16];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t K = p.K, KB = (K + 127) / 128;
  const int nchunk = (int)(FMT == kNormFp8b ? KB * 16 : (K + 7) / 8);
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    double sum = 0.0;
    for (int c = t; c < nchunk; c += 1024) {
      const Bytes16 h = load_sum(p, row, c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double v = (double)value_of(h, j);
        sum = __builtin_fma(v, v, sum);
      }
    }
    sum = wave_sum(sum);
    __syncthreads();  // the row before is done with sums and tops
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    sum = sums[0];
#pragma unroll
    for (int w = 1; w < 16; ++w) sum += sums[w];
    const float r = norm_factor(p, sum);
    const uint16_t* hr = p.residual ? p.h + row * p.ldh : p.x + row * p.ldx;
    auto load = [&](int c, Bytes16& h, Bytes16& g) __attribute__((always_inline)) {
      const int64_t k0 = (int64_t)c * 8;
      h = load_row8(hr + k0, K - k0);
      g = load_weight(p, k0);
    };
    float s = 0.0f;
    if (FMT == kNormInt8) {
      uint32_t top = 0;
      for (int c = t; c < nchunk; c += 1024) {
        Bytes16 h, g;
        load(c, h, g);
        top = max(top, chunk_max(h, g, r, K - (int64_t)c * 8));
      }
      top = wave_max_u32(top);
      if (lane == 0) tops[wave] = top;
      __syncthreads();
      top = tops[0];
#pragma unroll
      for (int w = 1; w < 16; ++w) top = max(top, tops[w]);
      s = __uint_as_float(top) / 127.0f;
      if (t == 0) reinterpret_cast<float*>(p.scale)[row] = s;
    }
    for (int c = t; c < nchunk; c += 1024) {
      Bytes16 h, g;
      load(c, h, g);
      write_chunk<FMT>(p, row, c, h, g, r, s);
    }
  }
}

template <int FMT, int CPL, int WPR>
static void launch(const NormArgs& p, hipStream_t stream) {
  constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;
  const int64_t groups = ceil_div(p.M, kRows);
  hipLaunchKernelGGL((rms_norm_kernel<FMT, CPL, WPR>), dim3((unsigned)std::min<int64_t>(groups, 2048)),
                     dim3(WPR >= 4 ? WPR * kWave : 256), 0, stream, p);
}

// Few rows: as many wavefronts a row as its chunks fill (64 x 4096 to INT8 4.2 us, with two
// chunks a lane 5.2). Many: more chunks a lane, so that fewer wavefronts meet at a barrier
// for each row (8192 x 7168 101 us, with a wavefront for every 64 chunks 127; 1024 x 7168
// 22.4 both ways), and no more than a row has (1237 x 4097 to E4M3 16.3 with three a lane,
// 17.6 with four; the third is nearly empty there, 4096 columns take 13.2).
template <int FMT>
static hipError_t launch_format(const NormArgs& p, hipStream_t stream) {
  const int64_t chunks = FMT == kNormFp8b ? ceil_div(p.K, 128) * 16 : ceil_div(p.K, 8);
  if (p.M > 512 && chunks <= 2 * 64) {
    if (chunks <= 64) launch<FMT, 1, 1>(p, stream);
    else launch<FMT, 2, 1>(p, stream);
  } else if (chunks <= 4 * 64) {
    launch<FMT, 1, 4>(p, stream);
  } else if (p.M > 512 && chunks <= 16 * 64) {
    if (chunks <= 8 * 64) launch<FMT, 2, 4>(p, stream);
    else if (chunks <= 12 * 64) launch<FMT, 3, 4>(p, stream);
    else launch<FMT, 4, 4>(p, stream);
  } else if (chunks <= 8 * 64) {
    launch<FMT, 1, 8>(p, stream);
  } else if (chunks <= 16 * 64) {
    launch<FMT, 1, 16>(p, stream);
  } else if (chunks <= 2 * 16 * 64) {
    launch<FMT, 2, 16>(p, stream);
  } else {
    hipLaunchKernelGGL((rms_norm_long_kernel<FMT>), dim3((unsigned)std::min<int64_t>(p.M, 2048)), dim3(1024), 0, stream, p);
  }
  return hipGetLastError();
}

hipError_t launch_rms_norm(int format, const NormArgs& p, hipStream_t stream) {
  if (p.M == 0) return hipSuccess;
  switch (format) {
    case kNormInt8: return launch_format<kNormInt8>(p, stream);
    case kNormFp8b: return launch_format<kNormFp8b>(p, stream);
    case kNormMx: return launch_format<kNormMx>(p, stream);
    default: return launch_format<kNormBf16>(p, stream);
  }
}

}  // namespace w8a8
