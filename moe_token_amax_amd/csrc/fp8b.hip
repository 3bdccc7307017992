// Block-scaled FP8 for gfx950: E4M3 activations with one fp32 scale per row and
// 128 values of K, E4M3 weights with one fp32 scale per 128 x 128 block, the
// product of the two in BF16, dense and grouped by expert.
//
// ("Qwen3.8-FP8 on Ascend 950: Why Weights Become MXFP8 at Load Time", Deep
// Dive 1: the checkpoint's contract, E4M3 weights with weight_scale_inv per
// 128 x 128 tile; here that form is multiplied as it is, with no resolve and no
// re-quantization.)
//
//   quant    s = fl(max|x| / 448), q = E4M3(fl(x / s)), half to even
//   product  y[m, n] = BF16(sum_b (s_x[m, b] s_w[n / 128, b]) P_b + bias[n]),
//            P_b = sum over the 128 k of block b of q_x[m, k] q_w[n, k]
//
// P_b is one MFMA of depth 128 with a zero accumulator; the scaled sum runs in
// fp32. The FP8 MFMA forms exact products, but adds the eight products of one
// 8-byte operand group after cutting each, towards zero, to a multiple of
// 2^(E - 13), E the largest sum of the two operands' exponents in the group
// (measured with in-bounds probes; groups add in fp32). That is below 2^-13 of
// the group's largest product per value, 1/32 of the half step of the BF16
// output, and the price of twice the BF16 matrix rate.
#include <algorithm>

#include "device_common.hpp"
#include "fp8b.hpp"
#include "launch.hpp"

namespace w8a8 {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp8BlockBytes = 2048;  // 16 rows x 128 k: two 1 KB pieces of 64 k

// fp32 -> BF16 with the hardware conversion: half to even, NaN stays NaN
__device__ __forceinline__ uint16_t to_bf16(float f) {
  const __bf16 b = (__bf16)f;
  return __builtin_bit_cast(uint16_t, b);
}

// ---------------------------------------------------------------------------
// quant
// ---------------------------------------------------------------------------
// max over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));  // row_half_mirror
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));  // row_mirror
  return v;
}

// Scale of a block from the bits of its largest magnitude. alg 1: the smallest
// power of two (at least 2^-126) not below amax / 448. NaN stays NaN.
__device__ __forceinline__ float block_scale(uint32_t amax_bits, int alg) {
  const float s = __uint_as_float(amax_bits) / 448.0f;
  if (alg == 0 || !(s > 0.0f) || !(s <= 3.402823466e38f)) return s;
  return __uint_as_float((__float_as_uint(s) + 0x7FFFFFu) & 0xFF800000u);
}

__device__ __forceinline__ float code_arg(float x, float s) {
  const float t = s > 0.0f ? x / s : 0.0f;
  return fminf(fmaxf(t, -448.0f), 448.0f);
}

template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t* src, int64_t n, float (&v)[8]) {
  if (VEC) {
    uint4 u = {0u, 0u, 0u, 0u};
    if (n >= 8) u = *reinterpret_cast<const uint4*>(src);  // VEC: the row's end is a multiple of 8
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? bf16_to_f32(src[j]) : 0.0f;
  }
}

// 16 lanes own one (row, block): 8 values a lane. A 256-thread workgroup takes
// 16 rows of one block at a time, so that the 16 scales of a block go out as
// one 64-byte piece of its [M] line.
constexpr int kQuantRows = 16;

template <int ACT, bool VEC>
__global__ __launch_bounds__(256) void fp8b_quant_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                         int64_t ldx, int alg, int KB, int per,
                                                         uint8_t* __restrict__ q, float* __restrict__ scale) {
  const int sub = threadIdx.x & 15;
  const int64_t row = (int64_t)blockIdx.x * kQuantRows + (threadIdx.x >> 4);
  if (row >= M) return;  // whole 16-lane rows leave together
  const int kb1 = min(KB, ((int)blockIdx.y + 1) * per);
  for (int kb = blockIdx.y * per; kb < kb1; ++kb) {
    const int64_t k0 = (int64_t)kb * kFp8Block + sub * 8;
    const uint16_t* src = x + row * ldx + k0;
    float v[8];
    load8<VEC>(src, K - k0, v);
    if (ACT == 1) {
      float u[8];
      load8<VEC>(src + K, K - k0, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = swiglu_fixed(v[j], u[j]);
    }
    uint32_t am = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) am = max(am, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    am = row_max_u32(am);
    const float s = block_scale(am, alg);
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(code_arg(v[0], s), code_arg(v[1], s), lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(code_arg(v[2], s), code_arg(v[3], s), lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(code_arg(v[4], s), code_arg(v[5], s), hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(code_arg(v[6], s), code_arg(v[7], s), hi, true);
    *reinterpret_cast<uint2*>(q + row * ((int64_t)KB * kFp8Block) + k0) = uint2{(uint32_t)lo, (uint32_t)hi};
    if (sub == 0) scale[(int64_t)kb * M + row] = s;
  }
}

hipError_t launch_fp8b_quant(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int act, int scale_alg,
                             uint8_t* q, float* scale, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  const int KB = (int)ceil_div(K, kFp8Block);
  const bool vec = K % 8 == 0 && ldx % 8 == 0 && ((uintptr_t)x & 15) == 0;
  const int64_t gx = ceil_div(M, kQuantRows);
  // enough workgroups to fill the chip, each with as many blocks as that leaves
  const int64_t gy = std::min<int64_t>(KB, std::max<int64_t>(1, ceil_div(2048, gx)));
  const int per = (int)ceil_div(KB, gy);
  const dim3 grid((unsigned)gx, (unsigned)ceil_div(KB, per));
  auto fn = act ? (vec ? fp8b_quant_kernel<1, true> : fp8b_quant_kernel<1, false>)
                : (vec ? fp8b_quant_kernel<0, true> : fp8b_quant_kernel<0, false>);
  hipLaunchKernelGGL(fn, grid, dim3(256), 0, stream, x, M, K, ldx, scale_alg, KB, per, q, scale);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Load-time layout of a weight: 2 KB blocks [e][n / 16][k / 128] of two 1 KB
// pieces; byte 16 l + j of piece h holds w[16 (n/16) + l % 16][128 (k/128) + 64 h +
// 16 (l / 16) + j], so that lane l's operand of the 16 x 16 x 128 MFMA is 16 bytes
// of each piece. N is zero-padded to 16, K to 128.
// ---------------------------------------------------------------------------
int64_t fp8b_packed_bytes(int64_t N, int64_t K) { return round_up(N, 16) * round_up(K, kFp8Block); }

__global__ __launch_bounds__(256) void fp8b_prepack_kernel(const uint8_t* __restrict__ w, int64_t E, int64_t N,
                                                           int64_t K, int64_t NB, int64_t KP, bool vec,
                                                           uint8_t* __restrict__ out) {
  const int64_t total = E * NB * KP * 64;  // 16-byte pieces; KP 64-deep pieces along K
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < total; g += (int64_t)gridDim.x * 256) {
    const int l = (int)(g & 63);
    const int64_t blk = g >> 6;
    const int64_t kp = blk % KP, nb = (blk / KP) % NB, e = blk / (KP * NB);
    const int64_t n = nb * 16 + (l & 15);
    const int64_t k0 = kp * 64 + (l >> 4) * 16;
    uint4 v = {0u, 0u, 0u, 0u};
    if (n < N && k0 < K) {
      const uint8_t* src = w + (e * N + n) * K + k0;
      if (vec) {
        v = *reinterpret_cast<const uint4*>(src);
      } else {
        uint32_t wd[4] = {0u, 0u, 0u, 0u};
        const int cnt = (int)min((int64_t)16, K - k0);
        for (int j = 0; j < cnt; ++j) wd[j >> 2] |= (uint32_t)src[j] << (8 * (j & 3));
        v = uint4{wd[0], wd[1], wd[2], wd[3]};
      }
    }
    *reinterpret_cast<uint4*>(out + g * 16) = v;
  }
}

hipError_t launch_fp8b_prepack(const uint8_t* w, int64_t E, int64_t N, int64_t K, void* packed,
                               hipStream_t stream) {
  const int64_t NB = ceil_div(N, 16), KP = 2 * ceil_div(K, kFp8Block);
  const int64_t total = E * NB * KP * 64;
  const bool vec = K % 16 == 0 && ((uintptr_t)w & 15) == 0;
  const int64_t grid = std::min<int64_t>(ceil_div(total, 256), 1 << 20);
  hipLaunchKernelGGL(fp8b_prepack_kernel, dim3((unsigned)grid), dim3(256), 0, stream, w, E, N, K, NB, KP, vec,
                     reinterpret_cast<uint8_t*>(packed));
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
// 16 x 16 x 128: lane l holds 32 bytes of row (A) or column (B) l % 16; result
// lane l holds column l % 16, rows 4 (l / 16) + {0..3}. Which 32 of the 128 k a
// lane holds does not matter as long as A and B agree.
__device__ __forceinline__ f32x4 mfma_fp8(const i32x8& a, const i32x8& b) {
  const f32x4 z = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ i32x8 load_operand(const uint8_t* p0, const uint8_t* p1) {
  const i32x4 x = *reinterpret_cast<const i32x4*>(p0);
  const i32x4 y = *reinterpret_cast<const i32x4*>(p1);
  return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 16 rows x 64 columns a workgroup, one 16-column block a wavefront, operands
// straight from global memory. The grouped form finds its (expert, 16-row tile)
// in a schedule that every workgroup builds in LDS.
__global__ __launch_bounds__(256) void fp8b_gemm_kernel(Fp8bGemm p) {
  __shared__ int64_t row_off[kMaxExperts + 1];
  __shared__ int tile_off[kMaxExperts + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int NB = (int)((p.N + 15) / 16), NS = (int)((p.N + kFp8Block - 1) / kFp8Block);
  int64_t row0 = (int64_t)blockIdx.x * 16, row_end = p.M;
  int e = 0;
  if (p.group_list) {
    const int E = (int)p.E;
    build_schedule<16>(p.group_list, E, row_off, tile_off);
    const int t = blockIdx.x;
    if (t >= tile_off[E]) return;
    int lo = 0, hi = E - 1;  // last expert whose tiles start at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile_off[mid] <= t) lo = mid; else hi = mid - 1;
    }
    e = lo;
    row0 = row_off[e] + (int64_t)(t - tile_off[e]) * 16;
    row_end = min(row_off[e + 1], p.M);
    if (row0 >= row_end) return;
  }
  const int nb = blockIdx.y * 4 + wave;
  if (nb >= NB) return;
  // rows past the tile's last read that row; they only feed rows never stored
  const int64_t m = min(row0 + (lane & 15), row_end - 1);
  int64_t ar = m;
  if (p.row_index) ar = max((int64_t)0, min((int64_t)p.row_index[m], p.a_rows - 1));
  const uint8_t* ap = p.a + ar * p.lda + (lane >> 4) * 16;
  const uint8_t* wp = p.w + ((int64_t)e * NB + nb) * p.KB * kFp8BlockBytes + lane * 16;
  const float* ws = p.w_scale + ((int64_t)e * NS + nb / 8) * p.KB;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t kb = 0; kb < p.KB; ++kb) {
    const i32x8 a = load_operand(ap + kb * 128, ap + kb * 128 + 64);
    const i32x8 b = load_operand(wp + kb * kFp8BlockBytes, wp + kb * kFp8BlockBytes + 1024);
    const f32x4 part = mfma_fp8(a, b);
    const float sx = p.a_scale[kb * p.a_rows + ar];  // of row lane % 16
    const float sw = ws[kb];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      acc[t] = __builtin_fmaf(part[t], __shfl(sx, (lane >> 4) * 4 + t) * sw, acc[t]);
  }
  const int64_t n = (int64_t)nb * 16 + (lane & 15);
  if (n >= p.N) return;
  const float b = p.bias ? bf16_to_f32(p.bias[n]) : 0.0f;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t r = row0 + (lane >> 4) * 4 + t;
    if (r < row_end) p.y[r * p.ldy + n] = to_bf16(p.bias ? acc[t] + b : acc[t]);
  }
}

int64_t fp8b_sched_bytes(int64_t E) { return group_sched_bytes(E); }

hipError_t launch_fp8b_gemm(const Fp8bGemm& p, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  const int64_t mt = ceil_div(p.M, 16) + (p.group_list ? p.E : 0);
  hipLaunchKernelGGL(fp8b_gemm_kernel, dim3((unsigned)mt, (unsigned)ceil_div(p.N, 64)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace w8a8
