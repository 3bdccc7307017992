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
// the group's largest product per value, which a BF16 output does not feel; where
// the output is quantized again (an expert's W13), its error grows to 1.6 times that
// of exact products, so EXACT tiles multiply the codes as BF16, at half the rate.
#include <algorithm>
#include <type_traits>

#include "bf16_io.hpp"
#include "device_common.hpp"
#include "epilogue.hpp"
#include "fp8_codes.hpp"
#include "fp8b.hpp"
#include "launch.hpp"

namespace w8a8 {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp8BlockBytes = 2048;  // 16 rows x 128 k: two 1 KB pieces of 64 k

// ---------------------------------------------------------------------------
// Schedule of a grouped product: int32 count (256 bytes), then int4 {expert,
// first row, rows, 0} for every tile of at most kTileRows rows of one expert,
// in expert order.
// ---------------------------------------------------------------------------
constexpr int kTileRows = 128;

int64_t fp8b_max_tiles(int64_t R, int64_t E) { return R / kTileRows + std::min(R, E); }
int64_t fp8b_sched_bytes(int64_t R, int64_t E) { return 256 + 16 * fp8b_max_tiles(R, E); }
// column groups of a row tile
constexpr int kGroupedNBW = 2, kSpreadTiles = 64;
static int64_t grouped_columns(int64_t N) { return ceil_div(N, 128 * kGroupedNBW); }
int64_t fp8b_grid_tiles(int64_t R, int64_t E, int64_t N) {
  return round_up(fp8b_max_tiles(R, E), 8) * grouped_columns(N);
}

struct Schedule {
  const int64_t* group_list;
  int E;  // at most 1024
  int64_t R;
  int* count;
  int4* tiles;
};

static Schedule schedule_of(const int64_t* group_list, int64_t E, int64_t R, void* ws) {
  return Schedule{group_list, (int)E, R, reinterpret_cast<int*>(ws),
                  reinterpret_cast<int4*>(reinterpret_cast<char*>(ws) + 256)};
}

// by a workgroup of 256 threads, four experts each
__device__ __forceinline__ void write_schedule(const Schedule& p) {
  __shared__ int64_t wrows[4];
  __shared__ int wtiles[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // counts past R are a caller error: such rows own no tile
  int64_t n[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    n[i] = 4 * tid + i < p.E ? min(max(p.group_list[4 * tid + i], (int64_t)0), p.R) : 0;
    sum += n[i];
  }
  int64_t ri = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(ri, d, 64);
    if (lane >= d) ri += o;
  }
  if (lane == 63) wrows[wave] = ri;
  __syncthreads();
  for (int w = 0; w < wave; ++w) ri += wrows[w];
  ri -= sum;
  int64_t row0[4];
  int t = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    row0[i] = min(ri, p.R);
    ri += n[i];
    n[i] = min(n[i], p.R - row0[i]);
    t += (int)((n[i] + kTileRows - 1) / kTileRows);
  }
  int ti = t;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(ti, d, 64);
    if (lane >= d) ti += o;
  }
  if (lane == 63) wtiles[wave] = ti;
  __syncthreads();
  for (int w = 0; w < wave; ++w) ti += wtiles[w];
  if (tid == 255) *p.count = ti;
  ti -= t;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    for (int64_t r = 0; r < n[i]; r += kTileRows)
      p.tiles[ti++] = int4{4 * tid + i, (int)(row0[i] + r), (int)min((int64_t)kTileRows, n[i] - r), 0};
}

__global__ __launch_bounds__(256) void fp8b_schedule_kernel(Schedule p) { write_schedule(p); }

hipError_t launch_fp8b_schedule(const int64_t* group_list, int64_t E, int64_t R, void* ws, hipStream_t stream) {
  hipLaunchKernelGGL(fp8b_schedule_kernel, dim3(1), dim3(256), 0, stream, schedule_of(group_list, E, R, ws));
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// quant
// ---------------------------------------------------------------------------
// ACT 1 quantizes swiglu_fixed, the INT8 quantizer's sequence of single roundings (its
// exponential is within 1.2 ulp): one SwiGLU for both, whose codes can be pinned bit by
// bit. It keeps the vector unit busy without a pause (16384 x 2048: 49 to 52 us, HBM 35).
// Of 10^8 codes 134 fall to the other side of a tie than 64 bits have them, with torch's
// exponential and division 136.
//
// 16 lanes own one (row, block): 8 values a lane. A 256-thread workgroup takes
// 16 rows of one block at a time, so that the 16 scales of a block go out as
// one 64-byte piece of its [M] line.
constexpr int kQuantRows = 16;

// SCHED: the first workgroup column writes a grouped product's schedule instead, which
// saves that launch where both have to run.
template <int ACT, bool SCHED>
__global__ __launch_bounds__(256) void fp8b_quant_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                         int64_t ldx, int alg, int KB, int per,
                                                         uint8_t* __restrict__ q, float* __restrict__ scale,
                                                         Schedule sched) {
  if (SCHED && blockIdx.x == 0) {
    if (blockIdx.y == 0) write_schedule(sched);
    return;
  }
  const int sub = threadIdx.x & 15;
  const int64_t row = ((int64_t)blockIdx.x - SCHED) * kQuantRows + (threadIdx.x >> 4);
  if (row >= M) return;  // whole 16-lane rows leave together
  const int kb1 = min(KB, ((int)blockIdx.y + 1) * per);
  for (int kb = blockIdx.y * per; kb < kb1; ++kb) {
    const int64_t k0 = (int64_t)kb * kFp8Block + sub * 8;
    const uint16_t* src = x + row * ldx + k0;
    float v[8], u[8];
    load8<ACT == 1>(src, K, K - k0, v, u);
    if (ACT == 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = swiglu_fixed(v[j], u[j]);
    }
    float s;
    const uint2 codes = quant_block(v, alg, s);
    *reinterpret_cast<uint2*>(q + row * ((int64_t)KB * kFp8Block) + k0) = codes;
    if (sub == 0) scale[(int64_t)kb * M + row] = s;
  }
}

template <int ACT, bool SCHED>
static hipError_t launch_quant(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int scale_alg, uint8_t* q,
                               float* scale, const Schedule& sched, hipStream_t stream) {
  const int KB = (int)ceil_div(K, kFp8Block);
  const int64_t gx = ceil_div(M, kQuantRows);
  // enough workgroups to fill the chip, each with as many blocks as that leaves
  const int64_t gy = std::min<int64_t>(KB, std::max<int64_t>(1, ceil_div(2048, gx)));
  const int per = (int)ceil_div(KB, gy);
  hipLaunchKernelGGL((fp8b_quant_kernel<ACT, SCHED>), dim3((unsigned)(gx + SCHED), (unsigned)ceil_div(KB, per)),
                     dim3(256), 0, stream, x, M, K, ldx, scale_alg, KB, per, q, scale, sched);
  return hipGetLastError();
}

hipError_t launch_fp8b_quant(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int act, int scale_alg,
                             uint8_t* q, float* scale, hipStream_t stream) {
  if (M == 0) return hipSuccess;
  return act ? launch_quant<1, false>(x, M, K, ldx, scale_alg, q, scale, Schedule{}, stream)
             : launch_quant<0, false>(x, M, K, ldx, scale_alg, q, scale, Schedule{}, stream);
}

hipError_t launch_fp8b_quant_schedule(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int scale_alg, uint8_t* q,
                                      float* scale, const int64_t* group_list, int64_t E, int64_t R, void* ws,
                                      hipStream_t stream) {
  return launch_quant<0, true>(x, M, K, ldx, scale_alg, q, scale, schedule_of(group_list, E, R, ws), stream);
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
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight E4M3 codes as BF16, exactly (an E4M3 value has 4 significant bits).
__device__ __forceinline__ bf16x8 codes_to_bf16(int lo, int hi) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return __builtin_bit_cast(bf16x8, uint4{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1),
                                          __builtin_bit_cast(uint32_t, p2), __builtin_bit_cast(uint32_t, p3)});
}

// Both MFMAs take the weight as the first operand: result lane l then holds
// row m = l % 16 of the activation block and columns 4 (l / 16) + {0..3} of the
// weight block, so that a lane has one activation scale per block and stores
// four neighbouring outputs. Which k of a block a lane supplies does not matter
// as long as both operands agree.
__device__ __forceinline__ f32x4 mfma_fp8(const i32x8& w, const i32x8& a) {
  const f32x4 z = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, z, 0, 0, 0, 0, 0, 0);
}

// Scaled sum of one 16 x 16 block. The empty asm keeps the result where it is
// computed: the compiler otherwise sinks the sums behind the next barrier and
// keeps every partial product of the step in registers (or in scratch) till then.
__device__ __forceinline__ void add_scaled(f32x4& acc, const f32x4& part, float s) {
#pragma unroll
  for (int t = 0; t < 4; ++t) acc[t] = __builtin_fmaf(part[t], s, acc[t]);
  asm volatile("" : "+v"(acc));
}

__device__ __forceinline__ i32x8 join(const i32x4& x, const i32x4& y) {
  return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}

#define W8A8_LDS __attribute__((address_space(3)))

template <int VM>
__device__ __forceinline__ void wait_vm_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Four neighbouring outputs of one row. EPI: the activation and the residual too, on the
// fp32 sums (kernels of their own: the plain ones keep their registers).
template <bool EPI>
__device__ __forceinline__ void store4(const Fp8bGemm& p, int64_t m, int64_t n, const f32x4& v) {
  if (n >= p.N) return;
  uint16_t* y = p.y + m * p.ldy + n;
  if (EPI) {
    const int left = (int)min((int64_t)4, p.N - n);
    float b[4], r[4];
    if (p.bias) load_bf16x4(p.bias + n, left, b);
    if (p.residual) load_bf16x4(p.residual + m * p.ldr + n, left, r);
    uint16_t o[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float a = activate(p.act, p.bias ? v[t] + b[t] : v[t]);
      o[t] = to_bf16(p.residual ? a + r[t] : a);
    }
    if (left == 4) {
      *reinterpret_cast<Bytes8*>(y) = Bytes8{{o[0] | ((uint32_t)o[1] << 16), o[2] | ((uint32_t)o[3] << 16)}};
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t < left) y[t] = o[t];
    }
    return;
  }
  if (n + 4 <= p.N) {
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.bias) {
      const Bytes8 u = *reinterpret_cast<const Bytes8*>(p.bias + n);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        b[2 * t] = __uint_as_float(u.w[t] << 16);
        b[2 * t + 1] = __uint_as_float(u.w[t] & 0xFFFF0000u);
      }
    }
    uint16_t o[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) o[t] = to_bf16(p.bias ? v[t] + b[t] : v[t]);
    *reinterpret_cast<Bytes8*>(y) = Bytes8{{o[0] | ((uint32_t)o[1] << 16), o[2] | ((uint32_t)o[3] << 16)}};
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (n + t < p.N) y[t] = to_bf16(p.bias ? v[t] + bf16_to_f32(p.bias[n + t]) : v[t]);
  }
}

// MB x NJ blocks of sums (this lane: rows row0 + 16 m + lane % 16 of `rows`, four columns of
// block nb + j) into y. EPI, all columns there: one piece of code for each activation, and
// what is loaded is there before a group of rows is stored (loads and stores are counted
// as one, so that a wait for a residual is one for every store before it; with a load and
// the choices at each output the wide tiles of 8192 x 4096 x 7168 with GELU and residual
// took 252 us, now 217; 208 without either).
template <bool EPI, int MB, int NJ>
__device__ __forceinline__ void store_blocks(const Fp8bGemm& p, int64_t row0, int rows, int64_t nb, int lane,
                                             const f32x4 (&acc)[MB][NJ]) {
  const int64_t n0 = nb * 16 + (lane >> 4) * 4;
  if (EPI && (nb + NJ) * 16 <= p.N) {  // wave-uniform
    constexpr int G = MB * NJ > 16 ? 8 / NJ : MB;  // (what registers are left)
    Bytes8 bias[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      bias[j] = Bytes8{{kNothing2, kNothing2}};
      if (p.bias) bias[j] = load_raw4<true>(p.bias + n0 + j * 16, 4);
    }
    for_act<false>(p.act, [&](auto ACT) __attribute__((always_inline)) {
#pragma unroll
      for (int m0 = 0; m0 < MB; m0 += G) {
        Bytes8 res[G][NJ];
#pragma unroll
        for (int m = 0; m < G; ++m)
#pragma unroll
          for (int j = 0; j < NJ; ++j) res[m][j] = Bytes8{{kNothing2, kNothing2}};
        if (p.residual) {
#pragma unroll
          for (int m = 0; m < G; ++m) {
            // (rows past the last load it)
            const uint16_t* src = p.residual + (row0 + min((m0 + m) * 16 + (lane & 15), rows - 1)) * p.ldr + n0;
#pragma unroll
            for (int j = 0; j < NJ; ++j) res[m][j] = load_raw4<true>(src + j * 16, 4);
          }
        }
#pragma unroll
        for (int m = 0; m < G; ++m)
#pragma unroll
          for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(res[m][j].w[0]), "+v"(res[m][j].w[1]));
        if (m0 == 0) {
#pragma unroll
          for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(bias[j].w[0]), "+v"(bias[j].w[1]));
        }
#pragma unroll
        for (int m = 0; m < G; ++m) {
          const int r = (m0 + m) * 16 + (lane & 15);
          if (r < rows) {
            uint16_t* y = p.y + (row0 + r) * p.ldy + n0;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              float v[4];
#pragma unroll
              for (int t = 0; t < 4; ++t) v[t] = acc[m0 + m][j][t] + bf16_of(bias[j], t);
              activate4(decltype(ACT)::value, v);
              uint32_t o[4];
#pragma unroll
              for (int t = 0; t < 4; ++t) o[t] = to_bf16(v[t] + bf16_of(res[m][j], t));
              *reinterpret_cast<Bytes8*>(y + j * 16) = Bytes8{{o[0] | (o[1] << 16), o[2] | (o[3] << 16)}};
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    });
    return;
  }
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int r = m * 16 + (lane & 15);
    if (r < rows) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) store4<EPI>(p, row0 + r, n0 + j * 16, acc[m][j]);
    }
  }
}

// Streaming tile: up to 16 MB rows x 128 NBW columns over the whole K, eight
// wavefronts, one workgroup a CU. Wavefront w owns the NBW 16-column blocks
// nb0 + NBW w + j and takes their weights from global memory straight into
// registers (the packed layout is the operand layout), kAhead blocks of K
// ahead: every weight byte of the tile is read once and never passes through
// LDS. The activation codes, which all eight share, go through LDS one block of
// K at a time (four buffers, one barrier a block), widened to BF16 on the way if
// EXACT. EXACT multiplies the codes as BF16 (16x16x32, every product exact, half
// the matrix rate); otherwise the FP8 MFMA. Up to 32 rows the weights' stream hides
// the difference, past that the LDS carries as much as the MFMAs take: 256 experts of
// 4096 x 4096, 2 / 32 / 64 / 128 rows each, exact 699 / 752 / 839 / 1282 us, else 695 /
// 748 / 788 / 931 (6.2 to 4.6 TB/s).
template <int MB, int NBW, bool EXACT, bool EPI = false>
struct StreamTile {
  static constexpr int kAhead = 3, kSets = kAhead + 1;  // blocks of weights in flight
  static constexpr int kWaves = 8;
  static constexpr int kPieces = (2 * MB + kWaves - 1) / kWaves;   // 16-byte pieces a thread stages per block of K
  static constexpr int kABytes = MB * (EXACT ? 4096 : 2048);       // one buffer's codes
  static constexpr int kBufBytes = kABytes + MB * 16 * 4;          // and its scales
  static constexpr int kLdsBytes = 4 * kBufBytes;

  struct Stage {
    i32x4 a[kPieces];
    float s;
  };
  struct Weights {
    i32x4 v[NBW][2];
    float s;  // scale of the block (a load of its own kept in step: used in the step that
              // issues it, it would wait for every weight load before it)
  };

  __device__ __forceinline__ static void run(const Fp8bGemm& p, uint8_t* smem, int e, int64_t row0, int rows, int nb0) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int NB = (int)((p.N + 15) / 16), NS = (int)((p.N + kFp8Block - 1) / kFp8Block);
    const int KB = (int)p.KB;
    const int nbw = nb0 + wave * NBW;
    // sources of this thread's pieces: piece (m-block, half) = wave + 8 i, lane:
    // row l % 16, 16 bytes at l / 16. Rows past the tile read its last row; they
    // only feed outputs that are never stored.
    const uint8_t* ap[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int piece = wave + kWaves * i;
      const int r = min((piece >> 1) * 16 + (lane & 15), rows - 1);
      int64_t src = row0 + r;
      if (p.row_index) src = max((int64_t)0, min((int64_t)p.row_index[src], p.a_rows - 1));
      ap[i] = p.a + src * p.lda + (piece & 1) * 64 + (lane >> 4) * 16;
    }
    const float* sp;
    {
      int64_t src = row0 + min(tid, rows - 1);
      if (p.row_index) src = max((int64_t)0, min((int64_t)p.row_index[src], p.a_rows - 1));
      sp = p.a_scale + src;
    }
    const uint8_t* wp[NBW];
#pragma unroll
    for (int j = 0; j < NBW; ++j)  // blocks past the last read it; their outputs are never stored
      wp[j] = p.w + ((int64_t)e * NB + min(nbw + j, NB - 1)) * KB * kFp8BlockBytes;
    const uint32_t l16 = lane * 16;
    const float* wsp = p.w_scale + ((int64_t)e * NS + min(nbw, NB - 1) / 8) * KB;

    auto load_w = [&](Weights& w, int kb) __attribute__((always_inline)) {
      const int64_t k = min(kb, KB - 1);
#pragma unroll
      for (int j = 0; j < NBW; ++j) {
        const uint8_t* b = wp[j] + k * kFp8BlockBytes;  // wave-uniform
        w.v[j][0] = *reinterpret_cast<const i32x4*>(b + l16);
        w.v[j][1] = *reinterpret_cast<const i32x4*>(b + l16 + 1024);
      }
      w.s = wsp[k];
    };
    auto load_a = [&](Stage& st, int kb) __attribute__((always_inline)) {
      const int64_t k = min(kb, KB - 1);
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (2 * MB >= kWaves * (i + 1) || wave + kWaves * i < 2 * MB) st.a[i] = *reinterpret_cast<const i32x4*>(ap[i] + k * 128);
      if (tid < 16 * MB) st.s = sp[k * p.a_rows];
    };
    auto store_a = [&](const Stage& st, uint8_t* buf) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int piece = wave + kWaves * i;
        if (2 * MB >= kWaves * (i + 1) || piece < 2 * MB) {
          if (EXACT) {
            *reinterpret_cast<bf16x8*>(buf + (2 * piece) * 1024 + lane * 16) = codes_to_bf16(st.a[i][0], st.a[i][1]);
            *reinterpret_cast<bf16x8*>(buf + (2 * piece + 1) * 1024 + lane * 16) = codes_to_bf16(st.a[i][2], st.a[i][3]);
          } else {
            *reinterpret_cast<i32x4*>(buf + piece * 1024 + lane * 16) = st.a[i];
          }
        }
      }
      if (tid < 16 * MB) *reinterpret_cast<float*>(buf + kABytes + tid * 4) = st.s;
    };

    f32x4 acc[MB][NBW];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int j = 0; j < NBW; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // Operands come in pieces of two 16-byte registers: a 16-row block (FP8), or
    // half of its K (EXACT); kN pieces a step.
    constexpr int kH = EXACT ? 2 : 1, kN = MB * kH, kD = kN < 2 ? kN : 2;
    struct Frag {
      i32x4 v[2];
    };
    Frag f[4];
    auto read_a = [&](Frag& d, const uint8_t* buf, int i) __attribute__((always_inline)) {
      d.v[0] = *reinterpret_cast<const i32x4*>(buf + i * 2048 + l16);
      d.v[1] = *reinterpret_cast<const i32x4*>(buf + i * 2048 + 1024 + l16);
    };
    auto read_s = [&](const uint8_t* buf, int m) __attribute__((always_inline)) {
      return *reinterpret_cast<const float*>(buf + kABytes + (m * 16 + (lane & 15)) * 4);
    };
    // Step kb: weights in set kb % 4, activation in buffer kb % 4. The weights of
    // kb + 3 and the activation of kb + 3 are loaded; kb is multiplied, each operand
    // read kD pieces before its MFMAs (the first ones in the step before, so that no
    // wavefront waits for LDS right behind the barrier) and the scaled sums of row
    // block m - 1 after the MFMAs of m (the last block's in the next step); the
    // activation of kb + 2 goes to its buffer, last read in step kb - 2, and is read
    // from the end of step kb + 1 on, behind the barrier of step kb. Loads past the
    // last block of K read it again.
    Weights w[kSets];
    Stage st[2];
    f32x4 part[2][NBW];
    float sc[2] = {0.f, 0.f}, sn;
#pragma unroll
    for (int j = 0; j < NBW; ++j) part[1][j] = part[0][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    load_a(st[0], 0);
    load_a(st[1], 1);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_w(w[i], i);
    store_a(st[0], smem);
    load_a(st[0], 2);
    store_a(st[1], smem + kBufBytes);
    lds_barrier();
#pragma unroll
    for (int i = 0; i < kD; ++i) read_a(f[i], smem, i);
    sn = read_s(smem, 0);
    auto step = [&](int kb, auto STEP) __attribute__((always_inline)) {
      constexpr int I = decltype(STEP)::value;
      const uint8_t* buf = smem + I * kBufBytes;
      const uint8_t* next = smem + ((I + 1) % 4) * kBufBytes;
      load_a(st[(I + 1) & 1], kb + 3);
      load_w(w[(I + kAhead) % kSets], kb + kAhead);
      const auto& wk = w[I].v;
      const float sw = w[I].s;
      bf16x8 wb[NBW][4];
      if (EXACT) {
#pragma unroll
        for (int j = 0; j < NBW; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            wb[j][q] = codes_to_bf16(wk[j][q >> 1][2 * (q & 1)], wk[j][q >> 1][2 * (q & 1) + 1]);
      }
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        // MB row blocks a step: the partial sums alternate over the whole run
        constexpr int odd = (I * MB) & 1;
        f32x4 (&cur)[NBW] = part[(m + odd) & 1];
        f32x4 (&old)[NBW] = part[(m + odd + 1) & 1];
        float& sold = sc[(m + odd + 1) & 1];
        sc[(m + odd) & 1] = sn * sw;
        sn = m + 1 < MB ? read_s(buf, m + 1) : read_s(next, 0);
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          const int i = m * kH + h;
          read_a(f[(I * kN + i + kD) % 4], i + kD < kN ? buf : next, (i + kD) % kN);
          __builtin_amdgcn_sched_barrier(0);
          const Frag& a = f[(I * kN + i) % 4];
          if (EXACT) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int j = 0; j < NBW; ++j)
                cur[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][2 * h + q], __builtin_bit_cast(bf16x8, a.v[q]),
                                                                 h + q ? cur[j] : f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
          } else {
#pragma unroll
            for (int j = 0; j < NBW; ++j) cur[j] = mfma_fp8(join(wk[j][0], wk[j][1]), join(a.v[0], a.v[1]));
          }
          if (h == 0) {
#pragma unroll
            for (int j = 0; j < NBW; ++j) add_scaled(acc[(m + MB - 1) % MB][j], old[j], sold);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      store_a(st[I & 1], smem + ((I + 2) % 4) * kBufBytes);
      lds_barrier();
    };
    // One call site per register set (with a second one, a remainder loop, the
    // compiler indexes the sets at run time, in scratch), and exits rather than
    // skipped steps: a path that skips a step, though it cannot be taken, makes the
    // compiler's waits let fewer loads be in flight.
    for (int kb = 0;; kb += kSets) {
      step(kb, std::integral_constant<int, 0>{});
      if (kb + 1 >= KB) break;
      step(kb + 1, std::integral_constant<int, 1>{});
      if (kb + 2 >= KB) break;
      step(kb + 2, std::integral_constant<int, 2>{});
      if (kb + 3 >= KB) break;
      step(kb + 3, std::integral_constant<int, 3>{});
      if (kb + 4 >= KB) break;
    }
    // the last row block's sums (MB odd: in the set that the last step left)
    const int last = MB % 2 ? (KB - 1) & 1 : 1;
#pragma unroll
    for (int j = 0; j < NBW; ++j) add_scaled(acc[MB - 1][j], last ? part[1][j] : part[0][j], last ? sc[1] : sc[0]);

    store_blocks<EPI>(p, row0, rows, nbw, lane, acc);
  }
};

// tile height by the rows there are
template <int NBW, bool EXACT>
__device__ __forceinline__ void stream_tile(const Fp8bGemm& p, uint8_t* smem, int e, int64_t row0, int rows, int nb0) {
  if (rows <= 16) StreamTile<1, NBW, EXACT>::run(p, smem, e, row0, rows, nb0);
  else if (rows <= 32) StreamTile<2, NBW, EXACT>::run(p, smem, e, row0, rows, nb0);
  else if (rows <= 64) StreamTile<4, NBW, EXACT>::run(p, smem, e, row0, rows, nb0);
  else if (rows <= 96) StreamTile<6, NBW, EXACT>::run(p, smem, e, row0, rows, nb0);
  else StreamTile<8, NBW, EXACT>::run(p, smem, e, row0, rows, nb0);
}

// Grouped: every row tile times NT column groups; workgroup b runs on XCD b % 8.
// Few tiles: in order, so that every XCD has its share. From kSpreadTiles on a tile's
// column groups go to two XCDs (one if NT is odd), whose L2 they read the tile's codes
// through, 4 or 8 tiles at a time; us of a layer of 256 experts of 4096 x 2048, top 8,
// on 8 / 4 / 2 / 1 XCDs a tile: 16 tokens 392 / 383 / 370 / 362, 2048 tokens 1519 / 1500 /
// 1499 / 1514; 8 experts, 4096 tokens, top 2: 534 / 521 / 541 / 564.
template <int NBW, bool EXACT>
__global__ __launch_bounds__(512) void fp8b_grouped_kernel(Fp8bGemm p, int NT) {
  using T = StreamTile<8, NBW, EXACT>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::kLdsBytes];
  const int count = *reinterpret_cast<const int*>(p.ws);
  int t, c;
  if (count >= kSpreadTiles) {
    const int spread = NT % 2 ? 1 : 2;
    const int x = blockIdx.x % 8, j = blockIdx.x / 8, per = NT / spread;
    t = j / per * (8 / spread) + x / spread;
    c = x % spread + j % per * spread;
  } else {
    t = blockIdx.x / NT;
    c = blockIdx.x % NT;
  }
  if (t >= count) return;
  const int nb0 = c * 8 * NBW;
  const int4 tile = reinterpret_cast<const int4*>(reinterpret_cast<const char*>(p.ws) + 256)[t];
  stream_tile<NBW, EXACT>(p, smem, __builtin_amdgcn_readfirstlane(tile.x), __builtin_amdgcn_readfirstlane(tile.y),
                          __builtin_amdgcn_readfirstlane(tile.z), nb0);
}

// Dense: tiles of one height.
template <int MB, int NBW, bool EPI>
__global__ __launch_bounds__(512) void fp8b_dense_kernel(Fp8bGemm p) {
  using T = StreamTile<MB, NBW, false, EPI>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::kLdsBytes];
  const int64_t row0 = (int64_t)blockIdx.x * (MB * 16);
  T::run(p, smem, 0, row0, (int)min((int64_t)(MB * 16), p.M - row0), blockIdx.y * 8 * NBW);
}

// Wide tiles: 256 rows x 256 columns over the whole K on the FP8 MFMA, eight
// wavefronts (2 x 4, each 128 x 64), both operands through LDS by DMA. The L2 hands a
// CU about 32 bytes a clock: a block of K takes 2 x 32 KB for 2048 clocks of MFMA,
// against 48 KB for 1024 in the streaming tile, whose wavefronts also spend
// registers and issue on the copies.
//
// LDS: two stages of one block of K, each 32 pieces of 8 activation rows x 128
// bytes (whole cache lines; slot l of a piece holds row l / 8, 16-byte chunk
// (l % 8) ^ (l / 8), so that the 16 rows of an operand lie in different banks), 32
// pieces of packed weight and the rows' scales; and the weight scales of two tiles.
// Step kb: row blocks 0..5, then "own DMA of kb + 1 landed, own reads of kb done,
// s_barrier", the DMA of kb + 2 into the stage of kb, row blocks 6 and 7 with the
// first operands of kb + 1 read between them. So a stage's DMA has one whole step
// to land, and one barrier a step serves both directions. A workgroup walks over
// its tiles without a gap: the last two steps of a tile load the first two blocks
// of the next one, which land while the tile is stored.
//
// Measured on 8192 x 4096 x 7168: MFMAs alone (a copy of the kernel without copies,
// reads and sums) 140 us on zeros, 169 on normal data (the clock gives way to the
// power that the data takes), the sums 5 / 20, LDS reads 9 / 7, DMA 15 / 42, barriers
// 27 / 17.
template <bool EPI>
struct WideTile {
  static constexpr int kOperand = 32768;           // one operand of one stage
  static constexpr int kScaleBytes = 1280;         // 256 row scales (and what the last wavefront's DMA runs over)
  static constexpr int kStage = 2 * kOperand + kScaleBytes;
  static constexpr int kMaxKB = 1041;              // ceil(W8A8_MAX_K / 128)
  static constexpr int kLdsBytes = 2 * kStage + 4 * kMaxKB * 4;

  struct Where {
    int rows, nb0;  // rows, first column block; rows 0: no tile
    int64_t row0;
  };

  // next(): this workgroup's next tile. KB >= 2.
  template <class Next>
  __device__ __forceinline__ static void run(const Fp8bGemm& p, uint8_t* smem, Next next) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int NB = (int)((p.N + 15) / 16), NS = (int)((p.N + kFp8Block - 1) / kFp8Block);
    const int KB = (int)p.KB;
    const uint32_t l16 = lane * 16;
    float* const wscales = reinterpret_cast<float*>(smem + 2 * kStage);  // [2][2][KB]
    uint32_t aoff[4];        // this wavefront's four activation pieces: bytes from a
    const float* sbase;      // its rows' scales of block 0, the last of them
    int slast;
    const uint8_t* wp[2];    // its two weight blocks
    // Sources of tile t; its weight scales go to half `par` of wscales.
    auto sources = [&](const Where& t, int par) __attribute__((always_inline)) {
      // rows past the tile read its last
#pragma unroll
      for (int i = 0; i < 4; ++i)
        aoff[i] = (uint32_t)((t.row0 + min((wave * 4 + i) * 8 + (lane >> 3), t.rows - 1)) * p.lda +
                             (((lane & 7) ^ (lane >> 3)) * 16));
      sbase = p.a_scale + t.row0 + min(wave * 32, t.rows - 1);
      slast = max(t.rows - 1 - wave * 32, 0);
#pragma unroll
      for (int j = 0; j < 2; ++j)  // past the last block, that one (never stored)
        wp[j] = p.w + (int64_t)min(t.nb0 + wave * 2 + j, NB - 1) * KB * kFp8BlockBytes;
      for (int i = tid; i < 2 * KB; i += 512) {
        const int h = i >= KB;
        wscales[par * 2 * KB + i] = p.w_scale[(int64_t)min(t.nb0 / 8 + h, NS - 1) * KB + (h ? i - KB : i)];
      }
    };
    // Addresses are a wave-uniform base and a 32-bit lane offset; the empty asm keeps
    // the compiler from hoisting their sums into register pairs.
    auto dma = [&](int64_t k, int stage) __attribute__((always_inline)) {
      W8A8_LDS uint8_t* dst = (W8A8_LDS uint8_t*)smem + stage * kStage;
      const uint8_t* ab = p.a + k * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o = aoff[i];
        asm volatile("" : "+v"(o));
        __builtin_amdgcn_global_load_lds(ab + o, (W8A8_LDS void*)(dst + (wave * 4 + i) * 1024), 16, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t o = l16;
        asm volatile("" : "+v"(o));
        const uint8_t* wb = wp[j >> 1] + k * kFp8BlockBytes + (j & 1) * 1024;
        __builtin_amdgcn_global_load_lds(wb + o, (W8A8_LDS void*)(dst + kOperand + (wave * 4 + j) * 1024), 16, 0, 0);
      }
      uint32_t o = min(lane, slast) * 4;
      asm volatile("" : "+v"(o));
      __builtin_amdgcn_global_load_lds(reinterpret_cast<const uint8_t*>(sbase + k * p.a_rows) + o,
                                       (W8A8_LDS void*)(dst + 2 * kOperand + wave * 128), 4, 0, 0);
    };
    // operand of row block m (16 rows) of this wavefront, and of its column block j
    const uint32_t arow = (wm * 128 + (lane & 15)) * 128 + (((lane >> 4) ^ (lane & 7)) * 16);
    auto read_a = [&](i32x8& d, const uint8_t* st, int m) __attribute__((always_inline)) {
      d = join(*reinterpret_cast<const i32x4*>(st + m * 2048 + arow), *reinterpret_cast<const i32x4*>(st + m * 2048 + (arow ^ 64)));
    };
    auto read_b = [&](i32x8& d, const uint8_t* st, int j) __attribute__((always_inline)) {
      const uint8_t* b = st + kOperand + (wn * 4 + j) * 2048 + l16;
      d = join(*reinterpret_cast<const i32x4*>(b), *reinterpret_cast<const i32x4*>(b + 1024));
    };
    auto read_s = [&](const uint8_t* st, int m) __attribute__((always_inline)) {
      return *reinterpret_cast<const float*>(st + 2 * kOperand + (wm * 128 + m * 16 + (lane & 15)) * 4);
    };
    Where cur = next();
    if (!cur.rows) return;
    sources(cur, 0);
    dma(0, 0);
    dma(1, 1);
    wait_vm_barrier<9>();  // stage 0 (and the scales) there
    i32x8 a[3], b[4];
    float sn;  // the next row block's scale, not yet times the weight's
#pragma unroll
    for (int j = 0; j < 4; ++j) read_b(b[j], smem, j);
    read_a(a[0], smem, 0);
    read_a(a[1], smem, 1);
    sn = read_s(smem, 0);
    int stage = 0, par = 0;
    for (;;) {
      f32x4 acc[8][4], part[4];
      float sc = 0.f, so = 0.f;  // scales of this row block and of the one before
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) part[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      Where after{0, 0, 0};
      const float* wsw = wscales + (par * 2 + (wn >> 1)) * KB;
      // TAIL: the tile's last two steps, whose DMA is the next tile's first
      auto step = [&](int kb, auto TAIL) __attribute__((always_inline)) {
        const uint8_t* st = smem + stage * kStage;
        const uint8_t* nx = smem + (stage ^ 1) * kStage;
        const float sw = wsw[kb];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          so = sc;
          sc = sn * sw;  // before the next reads: behind them it would wait for them too
          __builtin_amdgcn_sched_barrier(0);
          if (m < 6) {
            read_a(a[(m + 2) % 3], st, m + 2);
            sn = read_s(st, m + 1);
          } else if (m == 6) {
            sn = read_s(st, 7);
            // own reads of this stage done, own DMA of the next one landed, everyone
            // there: the next stage may be read and this one refilled
            wait_vm_barrier<0>();
            if constexpr (decltype(TAIL)::value) {
              if (after.rows) dma(kb + 2 - KB, stage);
            } else {
              dma(kb + 2, stage);
            }
            read_a(a[2], nx, 0);
          } else {
            sn = read_s(nx, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // the sums trail their MFMAs by three, and stay there: right behind its
            // MFMA a sum waits for the whole latency, and so does the next MFMA
            const int d = (j + 1) % 4;
            add_scaled(acc[j < 3 ? (m + 7) % 8 : m][d], part[d], j < 3 ? so : sc);
            part[j] = mfma_fp8(b[j], a[m % 3]);
            if (m == 7) read_b(b[j], nx, j);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (m == 7) {
            // row block 0 of the next step is in a[2]: rotate to a[0], a[1]
            a[0] = a[2];
            read_a(a[1], nx, 1);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        stage ^= 1;
      };
      for (int kb = 0; kb + 2 < KB; ++kb) step(kb, std::false_type{});
      after = next();
      if (after.rows) sources(after, par ^ 1);
      for (int kb = KB - 2; kb < KB; ++kb) step(kb, std::true_type{});
#pragma unroll
      for (int j = 1; j < 4; ++j) add_scaled(acc[7][j], part[j], sc);
      // EPI: the lane number read here, not kept (with what follows from it) over the K loop
      int el = lane;
      if (EPI) {
        el = threadIdx.x & 63;
        asm volatile("" : "+v"(el));
      }
      store_blocks<EPI>(p, cur.row0 + wm * 128, cur.rows - wm * 128, cur.nb0 + wn * 4, el, acc);
      if (!after.rows) break;
      cur = after;
      par ^= 1;
    }
  }
};

// Dense: one workgroup a CU; XCD x (workgroups b with b % 8 == x) walks over its own
// contiguous eighth of the tiles, 8 rows of tiles at a time, so that the tiles it
// runs together share panels in its L2.
template <bool EPI>
__global__ __launch_bounds__(512) void fp8b_wide_kernel(Fp8bGemm p) {
  using T = WideTile<EPI>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::kLdsBytes];
  const int64_t MT = (p.M + 255) / 256, NT = (p.N + 255) / 256, total = MT * NT;
  const int64_t per = (total + 7) / 8, first = (blockIdx.x % 8) * per, end = min(first + per, total);
  int64_t t = first + blockIdx.x / 8;
  T::run(p, smem, [&]() __attribute__((always_inline)) {
    typename T::Where w{0, 0, 0};
    if (t < end) {
      const int64_t top = t / (8 * NT) * 8, gm = min((int64_t)8, MT - top), r = t % (8 * NT);
      w.row0 = (top + r % gm) * 256;
      w.rows = (int)min((int64_t)256, p.M - w.row0);
      w.nb0 = (int)(r / gm) * 16;
      t += gridDim.x / 8;
    }
    return w;
  });
}

// Decode (dense, few rows): the weight's stream, split over K inside the workgroup.
// A workgroup owns NBW 16-column blocks and 16 MB rows over the whole K; its eight
// wavefronts take every eighth block of K, with U blocks of weights and codes in
// flight each, straight from global memory into operand registers and each set
// refilled as soon as it is multiplied, and their sums meet in LDS in a fixed
// order. FUSED (few rows): x is BF16, and every workgroup quantizes the rows itself
// into LDS, behind its first weight loads, which saves the quantizer's launch.
// Bound by the weights' stream (us in a graph): 1 x 16384 x 7168 22.2 of codes (5.3 TB/s),
// 25.4 with the quantizer inside; 16 rows 23.1. With tens of rows by the L1: the 16 lanes
// of a quarter of a code load lie in 16 rows, a look-up for every 16 bytes; 64 x 4096 x
// 7168 take 21246 look-ups a CU, 8.9 us at one a clock, of 11.4 (its lines from the L2, at
// 32 bytes a clock, 6.2).
constexpr int kDecodeWaves = 8;
constexpr int64_t kFusedValues = 8192;  // M x K quantized by every workgroup, at most

template <int MB, int NBW, int U, bool FUSED, bool EPI>
__global__ __launch_bounds__(kDecodeWaves * 64) void fp8b_decode_kernel(Fp8bGemm p) {
  __shared__ f32x4 red[kDecodeWaves][MB * NBW][kWave];
  extern __shared__ __attribute__((aligned(16))) uint8_t qlds[];  // FUSED: codes [M][128 KB], scales [KB][M]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int NB = (int)((p.N + 15) / 16), KB = (int)p.KB, M = (int)p.M;
  const int nb0 = blockIdx.x * NBW, m0 = blockIdx.y * MB * 16;
  const uint32_t l16 = lane * 16;
  const uint8_t* wp[NBW];
#pragma unroll
  for (int j = 0; j < NBW; ++j)  // blocks past the last read it; their outputs are never stored
    wp[j] = p.w + (int64_t)min(nb0 + j, NB - 1) * KB * kFp8BlockBytes;
  const float* wsp = p.w_scale + (int64_t)(nb0 / 8) * KB;  // NBW divides 8: one block of scales
  int row[MB];  // rows past the last read it; they only feed outputs that are never stored
#pragma unroll
  for (int m = 0; m < MB; ++m) row[m] = min(m0 + m * 16 + (lane & 15), M - 1);

  i32x4 w[U][NBW][2], a[U][MB][2];
  float sx[U][MB], sw[U];
  // block k (clamped) into set u
  auto load_w = [&](int u, int kb) __attribute__((always_inline)) {
    const int64_t k = min(kb, KB - 1);
#pragma unroll
    for (int j = 0; j < NBW; ++j) {
      const uint8_t* b = wp[j] + k * kFp8BlockBytes;
      w[u][j][0] = *reinterpret_cast<const i32x4*>(b + l16);
      w[u][j][1] = *reinterpret_cast<const i32x4*>(b + l16 + 1024);
    }
    sw[u] = wsp[k];
  };
  auto load_a = [&](int u, int kb) __attribute__((always_inline)) {
    const int64_t k = min(kb, KB - 1);
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      if (FUSED) {
        const uint8_t* src = qlds + row[m] * (KB * 128) + k * 128 + (lane >> 4) * 16;
        a[u][m][0] = *reinterpret_cast<const i32x4*>(src);
        a[u][m][1] = *reinterpret_cast<const i32x4*>(src + 64);
        sx[u][m] = reinterpret_cast<const float*>(qlds + M * (KB * 128))[k * M + row[m]];
      } else {
        const uint8_t* src = p.a + row[m] * p.lda + k * 128 + (lane >> 4) * 16;
        a[u][m][0] = *reinterpret_cast<const i32x4*>(src);
        a[u][m][1] = *reinterpret_cast<const i32x4*>(src + 64);
        sx[u][m] = p.a_scale[k * p.a_rows + row[m]];
      }
    }
  };

#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!FUSED) load_a(u, wave + u * kDecodeWaves);
    load_w(u, wave + u * kDecodeWaves);
  }
  if constexpr (FUSED) {
    __builtin_amdgcn_sched_barrier(0);
    // as fp8b_quant_kernel: 16 lanes a (row, block)
    const uint16_t* x = reinterpret_cast<const uint16_t*>(p.a);
    const int sub = tid & 15;
    for (int b = tid >> 4; b < M * KB; b += kDecodeWaves * 4) {
      const int r = b / KB, kb = b % KB;
      const int64_t k0 = (int64_t)kb * kFp8Block + sub * 8;
      float v[8], none[8];
      load8<false>(x + r * p.lda + k0, 0, p.K - k0, v, none);
      float s;
      const uint2 q = quant_block(v, p.scale_alg, s);
      *reinterpret_cast<uint2*>(qlds + r * (KB * 128) + k0) = q;
      if (sub == 0) reinterpret_cast<float*>(qlds + M * (KB * 128))[kb * M + r] = s;
    }
    __syncthreads();
  }
  f32x4 acc[MB][NBW];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int j = 0; j < NBW; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto mul = [&](int u) __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const float s = sx[u][m] * sw[u];
#pragma unroll
      for (int j = 0; j < NBW; ++j) {
        const f32x4 part = mfma_fp8(join(w[u][j][0], w[u][j][1]), join(a[u][m][0], a[u][m][1]));
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[m][j][t] = __builtin_fmaf(part[t], s, acc[m][j][t]);
      }
    }
  };
  __builtin_amdgcn_sched_barrier(0);  // every first load in flight before the first product
  int kb0 = wave;
  // a set is refilled as soon as it is multiplied
  for (; kb0 + kDecodeWaves * U < KB; kb0 += kDecodeWaves * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (FUSED) load_a(u, kb0 + u * kDecodeWaves);
      mul(u);
      if (!FUSED) load_a(u, kb0 + (u + U) * kDecodeWaves);
      load_w(u, kb0 + (u + U) * kDecodeWaves);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (kb0 < KB) {
    if (FUSED) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_a(u, kb0 + u * kDecodeWaves);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb0 + u * kDecodeWaves >= KB) break;  // wave-uniform: clamped blocks add nothing
      mul(u);
    }
  }
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int j = 0; j < NBW; ++j) red[wave][m * NBW + j][lane] = acc[m][j];
  __syncthreads();
  if (wave >= MB * NBW) return;
  f32x4 sum = red[0][wave][lane];
#pragma unroll
  for (int v = 1; v < kDecodeWaves; ++v) sum += red[v][wave][lane];
  const int r = m0 + (wave / NBW) * 16 + (lane & 15);
  if (r < M) store4<EPI>(p, r, (int64_t)(nb0 + wave % NBW) * 16 + (lane >> 4) * 4, sum);
}

// Whether a BF16 x of M rows is quantized inside the decode kernel: every
// workgroup does all of it, which past kFusedValues costs more than the
// quantizer's launch (us in a graph, inside / launched: 1 x 7168 x 2048 5.3 / 6.9,
// 1 x 4096 x 7168 9.0 / 9.9, 2 x 7168 x 7168 14.4 / 14.4, 4 x 7168 x 7168 17.2 / 14.4).
bool fp8b_fused_ok(int64_t M, int64_t K) {
  return M >= 1 && M <= 16 && M * K <= kFusedValues;
}

// U: a wavefront's blocks of K, at most as many as registers hold (sets without a
// block of their own load the last one again)
template <int MB, int NBW, bool FUSED, bool EPI>
static void launch_decode(const Fp8bGemm& p, hipStream_t stream) {
  constexpr int kMost = MB * NBW >= 8 ? 2 : MB * NBW >= 4 ? 4 : 8;
  const int64_t blocks = ceil_div(p.KB, kDecodeWaves);
  auto fn = blocks <= 2 ? fp8b_decode_kernel<MB, NBW, 2, FUSED, EPI>
          : blocks <= 4 ? fp8b_decode_kernel<MB, NBW, std::min(4, kMost), FUSED, EPI>
                        : fp8b_decode_kernel<MB, NBW, kMost, FUSED, EPI>;
  hipLaunchKernelGGL(fn, dim3((unsigned)ceil_div(ceil_div(p.N, 16), NBW), (unsigned)ceil_div(p.M, 16 * MB)),
                     dim3(kDecodeWaves * 64), FUSED ? (size_t)(p.M * p.KB * (kFp8Block + 4)) : 0, stream, p);
}

// whether the epilogue is more than a bias
static bool fp8b_epilogue(const Fp8bGemm& p) { return p.act != W8A8_ACT_NONE || p.residual; }

// whether pairs of column blocks reach a workgroup a CU at most (1 x 16384 x 7168: 28.9
// us one by one, 26.7 in pairs)
static bool fused_pairs(int64_t N) { return ceil_div(N, 16) > 256; }

hipError_t launch_fp8b_linear_fused(const Fp8bGemm& p, hipStream_t stream) {
  const bool pairs = fused_pairs(p.N);
  if (fp8b_epilogue(p)) {
    if (pairs) launch_decode<1, 2, true, true>(p, stream);
    else launch_decode<1, 1, true, true>(p, stream);
  } else {
    if (pairs) launch_decode<1, 2, true, false>(p, stream);
    else launch_decode<1, 1, true, false>(p, stream);
  }
  return hipGetLastError();
}

// Kernel of a dense product. Tall and wide tiles read operands less often, small ones
// give every CU work; which wins is read off measured times (microseconds; weights
// from memory; 1 to 1024 rows by 256 to 32768 columns, K 512 to 16384): a launch,
// `round` for every round of the chip (256 workgroups; 512 where two fit a CU) and
// per block of K `full` a round, but at least `first`. Over these sizes the choice
// is 1 % slower than the best kernel of each size in the mean, 26 % at worst.
//   us, best of the decode kernels / of the others:
//     rows x columns, K 7168:  1 x 4096 7.9 / 30   64 x 4096 14 / 33   64 x 16384 43 / 42
//                              333 x 1000 18 / 25  1024 x 4096 141 / 71
//     K 512:                   1 x 4096 3.1 / 4.3  64 x 4096 4.8 / 5.0  64 x 16384 12 / 6.3
enum DenseKernel { kDecode16, kDecode16x32, kDecode32, kDecode64, kTile32, kTile64, kTile64x256, kTile128, kTile256 };

struct Fp8bCost {
  DenseKernel kernel;
  int rows, cols;
  double launch, round, first, full;
  bool two;  // workgroups fit a CU
};

static const Fp8bCost& cheapest(const Fp8bGemm& p) {
  static constexpr Fp8bCost kCosts[] = {
      {kDecode16, 16, 16, 1.2, 1.7, 0.08, 0.09, false},    {kDecode16x32, 16, 32, 1.9, 1.0, 0.08, 0.12, false},
      {kDecode32, 32, 32, 1.5, 1.4, 0.14, 0.20, false},    {kDecode64, 64, 32, 2.4, 2.7, 0.24, 0.28, false},
      {kTile32, 32, 128, 3.9, 0.0, 0.46, 1.37, true},      {kTile64, 64, 128, 4.1, 0.0, 0.54, 1.55, true},
      {kTile64x256, 64, 256, 0.0, 4.5, 0.09, 0.77, false}, {kTile128, 128, 256, 5.3, 4.6, 1.08, 0.85, false},
      {kTile256, 256, 256, 13.0, 1.2, 0.09, 1.44, false}};
  const Fp8bCost* best = &kCosts[kTile128];
  double least = 1e30;
  for (const Fp8bCost& c : kCosts) {
    // the wide tile's pipeline is two blocks deep and its row offsets have 32 bits
    if (c.kernel == kTile256 && (p.KB < 2 || p.a_rows * p.lda >= (int64_t)1 << 32)) continue;
    if (c.kernel < kTile32 && p.M > 65535 * 16) continue;  // their rows are the grid's second dimension
    const int64_t n = ceil_div(p.M, c.rows) * ceil_div(p.N, c.cols);
    const double rounds = c.two ? n / 512.0 : (double)ceil_div(n, 256);
    const double us = c.launch + rounds * c.round + p.KB * std::max(c.first, rounds * c.full);
    if (us < least) {
      least = us;
      best = &c;
    }
  }
  return *best;
}

void fp8b_tile(const Fp8bGemm& p, bool quant_inside, int32_t* rows, int32_t* cols) {
  if (quant_inside) {
    *rows = 16;
    *cols = fused_pairs(p.N) ? 32 : 16;
  } else {
    const Fp8bCost& c = cheapest(p);
    *rows = c.rows;
    *cols = c.cols;
  }
}

template <int MB, int NBW, bool EPI>
static void launch_dense_tiles(const Fp8bGemm& p, hipStream_t stream) {
  hipLaunchKernelGGL((fp8b_dense_kernel<MB, NBW, EPI>),
                     dim3((unsigned)ceil_div(p.M, MB * 16), (unsigned)ceil_div(p.N, 128 * NBW)), dim3(512), 0, stream, p);
}

template <bool EPI>
static hipError_t launch_dense(const Fp8bGemm& p, hipStream_t stream) {
  switch (cheapest(p).kernel) {
    case kDecode16: launch_decode<1, 1, false, EPI>(p, stream); break;
    case kDecode16x32: launch_decode<1, 2, false, EPI>(p, stream); break;
    case kDecode32: launch_decode<2, 2, false, EPI>(p, stream); break;
    case kDecode64: launch_decode<4, 2, false, EPI>(p, stream); break;
    case kTile32: launch_dense_tiles<2, 1, EPI>(p, stream); break;
    case kTile64: launch_dense_tiles<4, 1, EPI>(p, stream); break;
    case kTile64x256: launch_dense_tiles<4, 2, EPI>(p, stream); break;
    case kTile128: launch_dense_tiles<8, 2, EPI>(p, stream); break;
    case kTile256: {
      const int64_t tiles = ceil_div(p.M, 256) * ceil_div(p.N, 256);
      hipLaunchKernelGGL(fp8b_wide_kernel<EPI>, dim3((unsigned)std::min<int64_t>(256, round_up(tiles, 8))), dim3(512), 0,
                         stream, p);
      break;
    }
  }
  return hipGetLastError();
}

hipError_t launch_fp8b_gemm(const Fp8bGemm& p, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  if (!p.group_list) return fp8b_epilogue(p) ? launch_dense<true>(p, stream) : launch_dense<false>(p, stream);
  constexpr int NBW = kGroupedNBW;
  const int64_t NT = grouped_columns(p.N);
  const dim3 grid((unsigned)fp8b_grid_tiles(p.M, p.E, p.N));
  if (p.exact) hipLaunchKernelGGL((fp8b_grouped_kernel<NBW, true>), grid, dim3(512), 0, stream, p, (int)NT);
  else hipLaunchKernelGGL((fp8b_grouped_kernel<NBW, false>), grid, dim3(512), 0, stream, p, (int)NT);
  return hipGetLastError();
}

}  // namespace w8a8
