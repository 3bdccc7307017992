// Products with a fused epilogue for gfx950: y = act(a w^T + bias) + residual.
//
//   INT8   acc exact in INT32; v = fl(fl(acc x_scale[m]) w_scale[n])
//   BF16   exact products, fp32 sums; SwiGLU of the weight's [gate | up] halves too
//
// The epilogue runs on the fp32 sums and rounds once, to the output. Both types share
// one layout, 1 KB blocks of 16 rows x 64 bytes in MFMA operand order (lane l holds row
// l % 16, bytes 16 (l / 16) .. + 16), and one set of kernels: per byte of K an INT8 MFMA
// does twice the products of a BF16 one in the same time.
//
// K runs in steps of 128 bytes (two 64-byte pieces). What of a's last step lies past K
// is zero, so that nothing behind a row (another row, a NaN) takes part.
#include <algorithm>
#include <type_traits>

#include "bf16_io.hpp"
#include "device_common.hpp"
#include "epilogue.hpp"
#include "fused.hpp"
#include "launch.hpp"

namespace w8a8 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Both operands 16 bytes a lane; the weight is the first, so that result lane l holds
// row m = l % 16 (l % 32) of a and 4 neighbouring columns in each 4 registers.
template <int TY>
struct Elem;

template <>
struct Elem<kFusedInt8> {
  using Acc4 = i32x4;
  using Acc16 = i32x16;
  __device__ __forceinline__ static Acc4 mma16(const i32x4& w, const i32x4& a, const Acc4& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, c, 0, 0, 0);
  }
  __device__ __forceinline__ static Acc16 mma32(const i32x4& w, const i32x4& a, const Acc16& c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(w, a, c, 0, 0, 0);
  }
};

template <>
struct Elem<kFusedBf16> {
  using Acc4 = f32x4;
  using Acc16 = f32x16;
  __device__ __forceinline__ static Acc4 mma16(const i32x4& w, const i32x4& a, const Acc4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, a), c, 0, 0,
                                                   0);
  }
  __device__ __forceinline__ static Acc16 mma32(const i32x4& w, const i32x4& a, const Acc16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, a), c, 0, 0,
                                                   0);
  }
};

__device__ __forceinline__ int bits_of(int32_t v) { return v; }
__device__ __forceinline__ int bits_of(float v) { return __float_as_int(v); }

constexpr int kStepBytes = 128;
constexpr int kPiece = 1024;  // 16 rows x 64 bytes

#define W8A8_LDS __attribute__((address_space(3)))

template <int VM>
__device__ __forceinline__ void wait_vm_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// ---------------------------------------------------------------------------
// a's rows in registers. 16 bytes at byte `off` of a row: whole pieces are loaded as
// they are; the piece that runs past the row's end is loaded from its last 16 bytes
// (in bounds, kbytes >= 16) and shifted into place by fix16 before it is used, and a
// piece behind the end becomes zero.
// ---------------------------------------------------------------------------
struct __attribute__((packed, aligned(1))) Row16 {
  i32x4 v;
};

__device__ __forceinline__ i32x4 load16(const uint8_t* row, uint32_t off, uint32_t last) {
  return reinterpret_cast<const Row16*>(row + min(off, last))->v;
}

// past = off - (kbytes - 16): bytes of the piece that were loaded too early
__device__ __forceinline__ i32x4 fix16(const i32x4& v, int past) {
  if (past <= 0) return v;
  const uint64_t lo = (uint32_t)v[0] | ((uint64_t)(uint32_t)v[1] << 32);
  const uint64_t hi = (uint32_t)v[2] | ((uint64_t)(uint32_t)v[3] << 32);
  uint64_t a = 0, b = 0;
  if (past < 8) {
    a = (lo >> (8 * past)) | (hi << (64 - 8 * past));
    b = hi >> (8 * past);
  } else if (past < 16) {
    a = hi >> (8 * (past - 8));
  }
  return i32x4{(int)(uint32_t)a, (int)(uint32_t)(a >> 32), (int)(uint32_t)b, (int)(uint32_t)(b >> 32)};
}

// ---------------------------------------------------------------------------
// epilogue
// ---------------------------------------------------------------------------
// the value in front of the activation, from a sum
__device__ __forceinline__ float scaled(const FusedGemm& p, int32_t acc, float xs, float ws) {
  return (float)acc * xs * ws;
}
__device__ __forceinline__ float scaled(const FusedGemm& p, float acc, float, float) { return acc; }

template <int TY>
__device__ __forceinline__ float row_scale(const FusedGemm& p, int64_t m) {
  return TY == kFusedInt8 ? p.a_scale[m] : 0.0f;
}

struct __attribute__((packed, aligned(4))) Floats4 {
  float v[4];
};

// Four neighbouring outputs (m, c .. c + 3) of `width`, from the sums of the weight rows
// n .. n + 3 (and of their partners `up`, rows n2 .. for SwiGLU).
template <int TY, class Acc>
__device__ __forceinline__ void emit4(const FusedGemm& p, int64_t m, int64_t c, int64_t width, const Acc& acc, float xs,
                                      const Acc* up) {
  if (c >= width) return;
  const int n = (int)min((int64_t)4, width - c);
  float b[4] = {0.f, 0.f, 0.f, 0.f}, b2[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f}, ws[4];
  if (p.bias) {
    load_bf16x4(p.bias + c, n, b);
    if (up) load_bf16x4(p.bias + width + c, n, b2);
  }
  if (p.residual) load_bf16x4(p.residual + m * p.ldr + c, n, r);
#pragma unroll
  for (int t = 0; t < 4; ++t) ws[t] = TY == kFusedInt8 ? p.w_scale[c + min(t, n - 1)] : 0.0f;
  float o[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    float v = scaled(p, acc[t], xs, ws[t]);
    if (p.bias) v = v + b[t];
    if (up) {
      float u = (float)(*up)[t];
      if (p.bias) u = u + b2[t];
      v = times_sigmoid(v, v) * u;
    } else {
      v = activate(p.act, v);
    }
    o[t] = p.residual ? v + r[t] : v;
  }
  if (p.f32) {
    float* y = reinterpret_cast<float*>(p.y) + m * p.ldy + c;
    if (n == 4) {
      *reinterpret_cast<Floats4*>(y) = Floats4{{o[0], o[1], o[2], o[3]}};
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t < n) y[t] = o[t];
    }
  } else {
    uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + m * p.ldy + c;
    uint32_t q[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) q[t] = to_bf16(o[t]);
    if (n == 4) {
      *reinterpret_cast<Bytes8*>(y) = Bytes8{{q[0] | (q[1] << 16), q[2] | (q[3] << 16)}};
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t < n) y[t] = (uint16_t)q[t];
    }
  }
}

__device__ __forceinline__ int64_t outputs_of(const FusedGemm& p) { return p.act == W8A8_ACT_SWIGLU ? p.N / 2 : p.N; }

// The 16 x 16 block nb of weight rows against the rows of m: this lane's four outputs.
// SwiGLU: nb even (gate), `up` the block after it.
template <int TY, class Acc>
__device__ __forceinline__ void emit_block(const FusedGemm& p, int64_t m, int64_t nb, int lane, const Acc& acc, float xs,
                                           const Acc* up) {
  const int64_t c = (up ? nb / 2 : nb) * 16 + (lane >> 4) * 4;
  emit4<TY>(p, m, c, outputs_of(p), acc, xs, up);
}

// ---------------------------------------------------------------------------
// Load-time layout of a BF16 weight: blocks [e][n-block][64 bytes of k], N padded to
// 32 (so that halves pair up whatever N is), K to 64, with zeros.
// ---------------------------------------------------------------------------
int64_t bf16_packed_bytes(int64_t N, int64_t K) { return round_up(N, 32) * round_up(K, 64) * 2; }

__global__ __launch_bounds__(256) void bf16_prepack_kernel(const uint16_t* __restrict__ w, int64_t E, int64_t N,
                                                           int64_t K, int64_t NB, int64_t KP, int pairs,
                                                           uint8_t* __restrict__ out) {
  const int64_t total = E * NB * KP * 64;  // 16-byte pieces
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < total; g += (int64_t)gridDim.x * 256) {
    const int l = (int)(g & 63);
    const int64_t blk = g >> 6;
    const int64_t kp = blk % KP, nb = (blk / KP) % NB, e = blk / (KP * NB);
    const int64_t half = N / 2;
    const int64_t r = (pairs ? nb / 2 : nb) * 16 + (l & 15);
    const int64_t n = pairs ? r + (nb & 1) * half : r;
    const int64_t k0 = kp * 32 + (l >> 4) * 8;
    Bytes16 v{};
    if (r < (pairs ? half : N) && k0 < K) {
      const uint16_t* src = w + (e * N + n) * K + k0;
      if (k0 + 8 <= K) {
        v = *reinterpret_cast<const Bytes16*>(src);
      } else {
        for (int j = 0; k0 + j < K; ++j) v.w[j / 2] |= (uint32_t)src[j] << (16 * (j & 1));
      }
    }
    *reinterpret_cast<uint4*>(out + g * 16) = uint4{v.w[0], v.w[1], v.w[2], v.w[3]};
  }
}

hipError_t launch_bf16_prepack(const uint16_t* w, int64_t E, int64_t N, int64_t K, bool pairs, void* packed,
                               hipStream_t stream) {
  const int64_t NB = round_up(N, 32) / 16, KP = 2 * ceil_div(K, 64);
  const int64_t grid = std::min<int64_t>(ceil_div(E * NB * KP * 64, 256), 1 << 20);
  hipLaunchKernelGGL(bf16_prepack_kernel, dim3((unsigned)grid), dim3(256), 0, stream, w, E, N, K, NB, KP, (int)pairs,
                     reinterpret_cast<uint8_t*>(packed));
  return hipGetLastError();
}

// Rows copied to whole, 16-byte aligned, zero-padded steps.
__global__ __launch_bounds__(256) void fused_copy_kernel(const uint8_t* __restrict__ a, int64_t M, int64_t lda,
                                                         int64_t kbytes, int64_t per, uint8_t* __restrict__ out) {
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < M * per; g += (int64_t)gridDim.x * 256) {
    const int64_t m = g / per, off = (g % per) * 16;
    const uint8_t* src = a + m * lda;
    i32x4 v = {0, 0, 0, 0};
    if (off + 16 <= kbytes) {
      v = reinterpret_cast<const Row16*>(src + off)->v;
    } else {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      for (int j = 0; j < 16 && off + j < kbytes; ++j) w[j >> 2] |= (uint32_t)src[off + j] << (8 * (j & 3));
      v = i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
    }
    *reinterpret_cast<i32x4*>(out + g * 16) = v;
  }
}

// ---------------------------------------------------------------------------
// Schedule of a grouped product: int32 count (256 bytes), then int4 {expert, first row,
// rows, 0} for every tile, in expert order: at most kTileRows rows of one expert.
// ---------------------------------------------------------------------------
constexpr int kTileRows = 128;
constexpr int kGroupedNBW = 2;

int64_t fused_max_tiles(int64_t R, int64_t E) { return R / kTileRows + std::min(R, E); }
int64_t fused_sched_bytes(int64_t R, int64_t E) { return 256 + 16 * fused_max_tiles(R, E); }
static int64_t grouped_columns(int64_t N) { return ceil_div(N, 128 * kGroupedNBW); }
int64_t fused_grid(int64_t R, int64_t E, int64_t N) { return round_up(fused_max_tiles(R, E), 8) * grouped_columns(N); }

// one workgroup of 256 threads, four experts each (E <= 1024)
__global__ __launch_bounds__(256) void fused_schedule_kernel(const int64_t* __restrict__ group_list, int E, int64_t R,
                                                             int* count, int4* tiles) {
  __shared__ int64_t wrows[4];
  __shared__ int wtiles[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // counts past R are a caller error: such rows own no tile
  int64_t n[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    n[i] = 4 * tid + i < E ? min(max(group_list[4 * tid + i], (int64_t)0), R) : 0;
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
    row0[i] = min(ri, R);
    ri += n[i];
    n[i] = min(n[i], R - row0[i]);
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
  if (tid == 255) *count = ti;
  ti -= t;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    for (int64_t r = 0; r < n[i]; r += kTileRows)
      tiles[ti++] = int4{4 * tid + i, (int)(row0[i] + r), (int)min((int64_t)kTileRows, n[i] - r), 0};
}

hipError_t launch_fused_schedule(const int64_t* group_list, int64_t E, int64_t R, void* ws, hipStream_t stream) {
  hipLaunchKernelGGL(fused_schedule_kernel, dim3(1), dim3(256), 0, stream, group_list, (int)E, R,
                     reinterpret_cast<int*>(ws), reinterpret_cast<int4*>(reinterpret_cast<char*>(ws) + 256));
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Streaming tile: up to 16 MB rows x 128 NBW columns over the whole K, eight
// wavefronts. Wavefront w owns the NBW 16-column blocks nb0 + NBW w + j and takes their
// weights from global memory straight into operand registers, kAhead steps ahead: every
// weight byte of the tile is read once and never passes through LDS. The rows, which
// all eight share, go through LDS one step at a time (four buffers, one barrier a step).
// ---------------------------------------------------------------------------
template <int TY, int MB, int NBW>
struct StreamTile {
  using Acc = typename Elem<TY>::Acc4;
  static constexpr int kAhead = 3, kSets = kAhead + 1;            // steps of weights in flight
  static constexpr int kWaves = 8;
  static constexpr int kPieces = (2 * MB + kWaves - 1) / kWaves;  // 16-byte pieces a thread stages per step
  static constexpr int kBufBytes = MB * 2 * kPiece;
  static constexpr int kLdsBytes = 4 * kBufBytes;

  struct Stage {
    i32x4 a[kPieces];
  };
  struct Weights {
    i32x4 v[NBW][2];
  };

  __device__ __forceinline__ static void run(const FusedGemm& p, uint8_t* smem, int e, int64_t row0, int rows, int nb0) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int NB = (int)p.NB, KP = (int)p.KP, KB = (KP + 1) / 2;
    const uint32_t last = (uint32_t)p.kbytes - 16;
    const int nbw = nb0 + wave * NBW;
    // sources of this thread's pieces: piece (m-block, half) = wave + 8 i, lane: row
    // l % 16, 16 bytes at l / 16. Rows past the tile read its last row; they only feed
    // outputs that are never stored.
    const uint8_t* ap[kPieces];
    uint32_t at[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int piece = wave + kWaves * i;
      const int r = min((piece >> 1) * 16 + (lane & 15), rows - 1);
      int64_t src = row0 + r;
      if (p.row_index) src = max((int64_t)0, min((int64_t)p.row_index[src], p.a_rows - 1));
      ap[i] = p.a + src * p.lda;
      at[i] = (piece & 1) * 64 + (lane >> 4) * 16;
    }
    const uint8_t* wp[NBW];
#pragma unroll
    for (int j = 0; j < NBW; ++j)  // blocks past the last read it; their outputs are never stored
      wp[j] = p.w + ((int64_t)e * NB + min(nbw + j, NB - 1)) * KP * kPiece;
    const uint32_t l16 = lane * 16;

    auto load_w = [&](Weights& w, int kb) __attribute__((always_inline)) {
      // an odd last piece is read twice: a is zero there
      const int64_t k0 = min(2 * kb, KP - 1), k1 = min(2 * kb + 1, KP - 1);
#pragma unroll
      for (int j = 0; j < NBW; ++j) {
        w.v[j][0] = *reinterpret_cast<const i32x4*>(wp[j] + k0 * kPiece + l16);
        w.v[j][1] = *reinterpret_cast<const i32x4*>(wp[j] + k1 * kPiece + l16);
      }
    };
    auto load_a = [&](Stage& st, int kb) __attribute__((always_inline)) {
      const uint32_t k = (uint32_t)min(kb, KB - 1) * kStepBytes;
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (2 * MB >= kWaves * (i + 1) || wave + kWaves * i < 2 * MB) st.a[i] = load16(ap[i], k + at[i], last);
    };
    auto store_a = [&](Stage& st, uint8_t* buf, int kb) __attribute__((always_inline)) {
      if (kb >= KB - 1) {  // the last step (or a copy of it)
        const int past = (KB - 1) * kStepBytes - (int)last;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) st.a[i] = fix16(st.a[i], past + (int)at[i]);
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int piece = wave + kWaves * i;
        if (2 * MB >= kWaves * (i + 1) || piece < 2 * MB)
          *reinterpret_cast<i32x4*>(buf + piece * kPiece + l16) = st.a[i];
      }
    };

    Acc acc[MB][NBW];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int j = 0; j < NBW; ++j) acc[m][j] = Acc{0, 0, 0, 0};

    constexpr int kD = MB < 2 ? MB : 2;
    struct Frag {
      i32x4 v[2];
    };
    Frag f[4];
    auto read_a = [&](Frag& d, const uint8_t* buf, int m) __attribute__((always_inline)) {
      d.v[0] = *reinterpret_cast<const i32x4*>(buf + m * 2 * kPiece + l16);
      d.v[1] = *reinterpret_cast<const i32x4*>(buf + m * 2 * kPiece + kPiece + l16);
    };
    // Step kb: weights in set kb % 4, rows in buffer kb % 4. The weights of kb + 3 and the
    // rows of kb + 3 are loaded; kb is multiplied, each operand read kD row blocks before
    // its MFMAs (the first ones in the step before, so that no wavefront waits for LDS
    // right behind the barrier); the rows of kb + 2 go to their buffer, last read in step
    // kb - 2, and are read from the end of step kb + 1 on, behind the barrier of step kb.
    // Loads past the last step read it again.
    Weights w[kSets];
    Stage st[2];
    load_a(st[0], 0);
    load_a(st[1], 1);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_w(w[i], i);
    store_a(st[0], smem, 0);
    load_a(st[0], 2);
    store_a(st[1], smem + kBufBytes, 1);
    lds_barrier();
#pragma unroll
    for (int i = 0; i < kD; ++i) read_a(f[i], smem, i);
    auto step = [&](int kb, auto STEP) __attribute__((always_inline)) {
      constexpr int I = decltype(STEP)::value;
      const uint8_t* buf = smem + I * kBufBytes;
      const uint8_t* next = smem + ((I + 1) % 4) * kBufBytes;
      load_a(st[(I + 1) & 1], kb + 3);
      load_w(w[(I + kAhead) % kSets], kb + kAhead);
      const auto& wk = w[I].v;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        read_a(f[(I * MB + m + kD) % 4], m + kD < MB ? buf : next, (m + kD) % MB);
        __builtin_amdgcn_sched_barrier(0);
        const Frag& a = f[(I * MB + m) % 4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int j = 0; j < NBW; ++j) acc[m][j] = Elem<TY>::mma16(wk[j][q], a.v[q], acc[m][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      store_a(st[I & 1], smem + ((I + 2) % 4) * kBufBytes, kb + 2);
      lds_barrier();
    };
    // one call site per register set, and exits rather than skipped steps (see the
    // block-scaled tile: remainders put the sets in scratch, skipped steps shorten the
    // waits)
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
    const bool swiglu = p.act == W8A8_ACT_SWIGLU;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int r = m * 16 + (lane & 15);
      if (r < rows) {
        const float xs = row_scale<TY>(p, row0 + r);
        if (NBW == 2 && swiglu) {
          emit_block<TY>(p, row0 + r, nbw, lane, acc[m][0], xs, &acc[m][NBW - 1]);
        } else {
#pragma unroll
          for (int j = 0; j < NBW; ++j) emit_block<TY, Acc>(p, row0 + r, nbw + j, lane, acc[m][j], xs, nullptr);
        }
      }
    }
  }
};

// tile height by the rows there are
template <int TY, int NBW>
__device__ __forceinline__ void stream_tile(const FusedGemm& p, uint8_t* smem, int e, int64_t row0, int rows, int nb0) {
  if (rows <= 16) StreamTile<TY, 1, NBW>::run(p, smem, e, row0, rows, nb0);
  else if (rows <= 32) StreamTile<TY, 2, NBW>::run(p, smem, e, row0, rows, nb0);
  else if (rows <= 64) StreamTile<TY, 4, NBW>::run(p, smem, e, row0, rows, nb0);
  else if (rows <= 96) StreamTile<TY, 6, NBW>::run(p, smem, e, row0, rows, nb0);
  else StreamTile<TY, 8, NBW>::run(p, smem, e, row0, rows, nb0);
}

// Grouped: every row tile times NT column groups; workgroup b runs on XCD b % 8. A
// tile's column groups go to two XCDs (one if NT is odd), whose L2 they read the tile's
// rows through, 4 or 8 tiles at a time.
constexpr int kSpreadTiles = 64;

template <int TY, int NBW>
__global__ __launch_bounds__(512) void fused_grouped_kernel(FusedGemm p, int NT) {
  using T = StreamTile<TY, 8, NBW>;
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
  const int4 tile = reinterpret_cast<const int4*>(reinterpret_cast<const char*>(p.ws) + 256)[t];
  stream_tile<TY, NBW>(p, smem, __builtin_amdgcn_readfirstlane(tile.x), __builtin_amdgcn_readfirstlane(tile.y),
                       __builtin_amdgcn_readfirstlane(tile.z), c * 8 * NBW);
}

// Dense: tiles of one height.
template <int TY, int MB, int NBW>
__global__ __launch_bounds__(512) void fused_dense_kernel(FusedGemm p) {
  using T = StreamTile<TY, MB, NBW>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::kLdsBytes];
  const int64_t row0 = (int64_t)blockIdx.x * (MB * 16);
  T::run(p, smem, 0, row0, (int)min((int64_t)(MB * 16), p.M - row0), blockIdx.y * 8 * NBW);
}

// ---------------------------------------------------------------------------
// Decode (dense, few rows): the weight's stream, split over K inside the workgroup. A
// workgroup owns NBW 16-column blocks and 16 MB rows over the whole K; its eight
// wavefronts take every eighth step, with U steps of weights and rows in flight each,
// straight from global memory into operand registers and each set refilled as soon as
// it is multiplied, and their sums meet in LDS in a fixed order.
// ---------------------------------------------------------------------------
constexpr int kDecodeWaves = 8;

template <int TY, int MB, int NBW, int U>
__global__ __launch_bounds__(kDecodeWaves * 64) void fused_decode_kernel(FusedGemm p) {
  using Acc = typename Elem<TY>::Acc4;
  __shared__ Acc red[kDecodeWaves][MB * NBW][kWave];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int NB = (int)p.NB, KP = (int)p.KP, KB = (KP + 1) / 2, M = (int)p.M;
  const uint32_t last = (uint32_t)p.kbytes - 16;
  const int nb0 = blockIdx.x * NBW, m0 = blockIdx.y * MB * 16;
  const uint32_t l16 = lane * 16, at = (lane >> 4) * 16;
  const uint8_t* wp[NBW];
#pragma unroll
  for (int j = 0; j < NBW; ++j)  // blocks past the last read it; their outputs are never stored
    wp[j] = p.w + (int64_t)min(nb0 + j, NB - 1) * KP * kPiece;
  const uint8_t* ap[MB];  // rows past the last read it; they only feed outputs that are never stored
#pragma unroll
  for (int m = 0; m < MB; ++m) ap[m] = p.a + (int64_t)min(m0 + m * 16 + (lane & 15), M - 1) * p.lda;

  i32x4 w[U][NBW][2], a[U][MB][2];
  // step k (clamped) into set u
  auto load_w = [&](int u, int kb) __attribute__((always_inline)) {
    const int64_t k0 = min(2 * kb, KP - 1), k1 = min(2 * kb + 1, KP - 1);
#pragma unroll
    for (int j = 0; j < NBW; ++j) {
      w[u][j][0] = *reinterpret_cast<const i32x4*>(wp[j] + k0 * kPiece + l16);
      w[u][j][1] = *reinterpret_cast<const i32x4*>(wp[j] + k1 * kPiece + l16);
    }
  };
  auto load_a = [&](int u, int kb) __attribute__((always_inline)) {
    const uint32_t k = (uint32_t)min(kb, KB - 1) * kStepBytes + at;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      a[u][m][0] = load16(ap[m], k, last);
      a[u][m][1] = load16(ap[m], k + 64, last);
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    load_a(u, wave + u * kDecodeWaves);
    load_w(u, wave + u * kDecodeWaves);
  }
  Acc acc[MB][NBW];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int j = 0; j < NBW; ++j) acc[m][j] = Acc{0, 0, 0, 0};
  auto mul = [&](int u, int kb) __attribute__((always_inline)) {
    if (kb == KB - 1) {  // wave-uniform
      const int past = (KB - 1) * kStepBytes - (int)last + (int)at;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        a[u][m][0] = fix16(a[u][m][0], past);
        a[u][m][1] = fix16(a[u][m][1], past + 64);
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < NBW; ++j) acc[m][j] = Elem<TY>::mma16(w[u][j][q], a[u][m][q], acc[m][j]);
  };
  __builtin_amdgcn_sched_barrier(0);  // every first load in flight before the first product
  int kb0 = wave;
  for (; kb0 + kDecodeWaves * U < KB; kb0 += kDecodeWaves * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mul(u, kb0 + u * kDecodeWaves);
      load_a(u, kb0 + (u + U) * kDecodeWaves);
      load_w(u, kb0 + (u + U) * kDecodeWaves);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (kb0 < KB) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb0 + u * kDecodeWaves >= KB) break;  // wave-uniform: clamped steps add nothing
      mul(u, kb0 + u * kDecodeWaves);
    }
  }
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int j = 0; j < NBW; ++j) red[wave][m * NBW + j][lane] = acc[m][j];
  __syncthreads();
  auto total = [&](int b) __attribute__((always_inline)) {
    Acc sum = red[0][b][lane];
#pragma unroll
    for (int v = 1; v < kDecodeWaves; ++v) sum += red[v][b][lane];
    return sum;
  };
  const bool swiglu = NBW == 2 && p.act == W8A8_ACT_SWIGLU;
  const int per = swiglu ? NBW / 2 : NBW;  // blocks of outputs beside each other
  if (wave >= MB * per) return;
  const int64_t r = m0 + (wave / per) * 16 + (lane & 15);
  if (r >= M) return;
  const float xs = row_scale<TY>(p, r);
  if (swiglu) {
    const Acc gate = total(wave * 2), up = total(wave * 2 + 1);
    emit_block<TY>(p, r, nb0, lane, gate, xs, &up);
  } else {
    emit_block<TY, Acc>(p, r, nb0 + wave % NBW, lane, total(wave), xs, nullptr);
  }
}

// ---------------------------------------------------------------------------
// Wide tiles: 256 rows x 256 columns over the whole K, eight wavefronts (2 x 4, each
// 128 x 64 as 4 x 2 blocks of the 32 x 32 MFMA), both operands through LDS by DMA.
//
// LDS: two stages of one step, each 32 pieces of 8 rows x 128 bytes of a (whole cache
// lines; slot l of a piece holds row l / 8, 16-byte chunk (l % 8) ^ (l / 8), so that the
// rows of an operand lie in different banks) and 32 pieces of packed weight; and 4 KB a
// wavefront through which the sums are turned into whole lines of y.
// Step kb, in four quarters of 32 bytes of K: the operands of a quarter are read while
// the one before is multiplied; before the last quarter's MFMAs "own DMA of kb + 1
// landed, own reads of kb done, s_barrier", then the DMA of kb + 2 into the stage of
// kb. A workgroup walks over its tiles without a gap: the last two steps of a tile load
// the first two of the next one, which land while the tile is stored.
// ---------------------------------------------------------------------------
static __device__ __align__(16) uint8_t zeros16[16];

template <int TY>
struct WideTile {
  using Acc = typename Elem<TY>::Acc16;
  static constexpr int kOperand = 32768;  // one operand of one stage
  static constexpr int kStage = 2 * kOperand;
  static constexpr int kTurn = 4096;      // a wavefront's room in the epilogue
  static constexpr int kLdsBytes = 2 * kStage + 8 * kTurn;

  struct Where {
    int rows, nb0;  // rows, first column block; rows 0: no tile
    int64_t row0;
  };

  // This wavefront's 32 x 32 block of sums (m, n): rows row0 + 32 of `rows`, weight rows
  // from block nb. Turned through LDS (16-byte chunk c of row r at c ^ (r % 8)), so that
  // a lane holds 8 neighbouring columns and four (SwiGLU: two) lanes a row.
  __device__ __forceinline__ static void store_block(const FusedGemm& p, uint8_t* turn, const Acc& acc, int64_t row0,
                                                     int rows, int nb) {
    const int lane = threadIdx.x & 63;
    if (rows <= 0) return;  // the same in every lane
    const int64_t width = outputs_of(p);
    const bool swiglu = p.act == W8A8_ACT_SWIGLU;
    uint8_t* mine = turn + (lane & 31) * 128;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      i32x4 v;
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = bits_of(acc[4 * g + t]);
      *reinterpret_cast<i32x4*>(mine + (((2 * g + (lane >> 5)) ^ (lane & 7)) * 16)) = v;
    }
    // the same wavefront reads it back: in order, no barrier
    __builtin_amdgcn_wave_barrier();
    auto read8 = [&](int r, int c8, float (&v)[8], float xs, const float (&ws)[8]) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const i32x4 u = *reinterpret_cast<const i32x4*>(turn + r * 128 + (((2 * c8 + h) ^ (r & 7)) * 16));
#pragma unroll
        for (int t = 0; t < 4; ++t)
          v[4 * h + t] = TY == kFusedInt8 ? scaled(p, (int32_t)u[t], xs, ws[4 * h + t]) : __int_as_float(u[t]);
      }
    };
    const int lanes = swiglu ? 2 : 4;                   // a row
    const int c8 = lane % lanes;
    const int64_t c = (int64_t)(swiglu ? nb / 2 : nb) * 16 + c8 * 8;
    const int64_t n = width - c;                        // columns there are
    float b[8], b2[8], ws[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int64_t ct = min(c + t, width - 1);
      b[t] = p.bias ? bf16_to_f32(p.bias[ct]) : 0.0f;
      b2[t] = p.bias && swiglu ? bf16_to_f32(p.bias[width + ct]) : 0.0f;
      ws[t] = TY == kFusedInt8 ? p.w_scale[ct] : 0.0f;
    }
    for (int r = lane / lanes; r < 32; r += 64 / lanes) {
      const int64_t m = row0 + r;
      const bool in = r < rows && n > 0;
      float v[8], u[8];
      const float xs = in ? row_scale<TY>(p, m) : 0.0f;
      read8(r, c8, v, xs, ws);
      if (swiglu) read8(r, c8 + 2, u, xs, ws);
      if (!in) continue;
      float res[8], none[8];
      if (p.residual) load8<false>(p.residual + m * p.ldr + c, 0, n, res, none);
      float o[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        float z = p.bias ? v[t] + b[t] : v[t];
        if (swiglu) z = times_sigmoid(z, z) * (p.bias ? u[t] + b2[t] : u[t]);
        else z = activate(p.act, z);
        o[t] = p.residual ? z + res[t] : z;
      }
      if (p.f32) {
        float* y = reinterpret_cast<float*>(p.y) + m * p.ldy + c;
        if (n >= 8) {
          *reinterpret_cast<Floats4*>(y) = Floats4{{o[0], o[1], o[2], o[3]}};
          *reinterpret_cast<Floats4*>(y + 4) = Floats4{{o[4], o[5], o[6], o[7]}};
        } else {
#pragma unroll
          for (int t = 0; t < 8; ++t)
            if (t < n) y[t] = o[t];
        }
      } else {
        uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + m * p.ldy + c;
        uint32_t q[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) q[t] = to_bf16(o[t]);
        if (n >= 8) {
          *reinterpret_cast<Bytes16*>(y) =
              Bytes16{{q[0] | (q[1] << 16), q[2] | (q[3] << 16), q[4] | (q[5] << 16), q[6] | (q[7] << 16)}};
        } else {
#pragma unroll
          for (int t = 0; t < 8; ++t)
            if (t < n) y[t] = (uint16_t)q[t];
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }

  // next(): this workgroup's next tile. At least two steps of K.
  template <class Next>
  __device__ __forceinline__ static void run(const FusedGemm& p, uint8_t* smem, Next next) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int NB = (int)p.NB, KP = (int)p.KP, KB = (KP + 1) / 2;
    const uint32_t l16 = lane * 16;
    const uint32_t chunk = ((lane & 7) ^ (lane >> 3)) * 16;
    const bool ragged = p.kbytes != (int64_t)KB * kStepBytes;
    const uint8_t* abase;    // the tile's first row
    uint32_t aoff[4];        // this wavefront's four pieces of a: bytes from abase
    const uint8_t* wp[2];    // its two weight blocks
    auto sources = [&](const Where& t) __attribute__((always_inline)) {
      abase = p.a + t.row0 * p.lda;
      // rows past the tile read its last
#pragma unroll
      for (int i = 0; i < 4; ++i)
        aoff[i] = (uint32_t)(min((wave * 4 + i) * 8 + (lane >> 3), t.rows - 1) * (uint32_t)p.lda + chunk);
#pragma unroll
      for (int j = 0; j < 2; ++j)  // past the last block, that one (never stored)
        wp[j] = p.w + (int64_t)min(t.nb0 + wave * 2 + j, NB - 1) * KP * kPiece;
    };
    // Addresses are a wave-uniform base and a 32-bit lane offset; the empty asm keeps
    // the compiler from hoisting their sums into register pairs.
    auto dma = [&](int k, int stage) __attribute__((always_inline)) {
      W8A8_LDS uint8_t* dst = (W8A8_LDS uint8_t*)smem + stage * kStage;
      const uint8_t* ab = abase + (int64_t)k * kStepBytes;
      if (ragged && k == KB - 1) {  // the same in every lane
        const bool in = (int64_t)k * kStepBytes + chunk < p.kbytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* src = in ? ab + aoff[i] : zeros16;
          __builtin_amdgcn_global_load_lds(src, (W8A8_LDS void*)(dst + (wave * 4 + i) * 1024), 16, 0, 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o = aoff[i];
          asm volatile("" : "+v"(o));
          __builtin_amdgcn_global_load_lds(ab + o, (W8A8_LDS void*)(dst + (wave * 4 + i) * 1024), 16, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t o = l16;
        asm volatile("" : "+v"(o));
        const uint8_t* wb = wp[j >> 1] + (int64_t)min(2 * k + (j & 1), KP - 1) * kPiece;
        __builtin_amdgcn_global_load_lds(wb + o, (W8A8_LDS void*)(dst + kOperand + (wave * 4 + j) * 1024), 16, 0, 0);
      }
    };
    // operands of quarter s: 32 rows (l % 32), 16 bytes at l / 32 of its 32
    const uint32_t ar = (wm * 128 + (lane & 31)) * 128, a7 = lane & 7;
    const uint32_t br = kOperand + ((wn * 4 + ((lane >> 4) & 1)) * 2) * kPiece + (lane & 15) * 16 + (lane >> 5) * 256;
    struct Ops {
      i32x4 a[4], b[2];
    };
    auto read = [&](Ops& d, const uint8_t* st, int s) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        d.b[j] = *reinterpret_cast<const i32x4*>(st + br + (j * 4 + (s >> 1)) * kPiece + (s & 1) * 512);
      const uint32_t slot = ((2 * s + (lane >> 5)) ^ a7) * 16;
#pragma unroll
      for (int i = 0; i < 4; ++i) d.a[i] = *reinterpret_cast<const i32x4*>(st + ar + i * 4096 + slot);
    };
    Where cur = next();
    if (!cur.rows) return;
    sources(cur);
    dma(0, 0);
    dma(1, 1);
    wait_vm_barrier<8>();  // stage 0 there
    Ops ops[2];
    read(ops[0], smem, 0);
    int stage = 0;
    for (;;) {
      Acc acc[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int t = 0; t < 16; ++t) acc[i][j][t] = 0;
      Where after{0, 0, 0};
      // TAIL: the tile's last two steps, whose DMA is the next tile's first
      auto step = [&](int kb, auto TAIL) __attribute__((always_inline)) {
        const uint8_t* st = smem + stage * kStage;
        const uint8_t* nx = smem + (stage ^ 1) * kStage;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const Ops& o = ops[s & 1];
          // A quarter's first products stand before the next one's reads: beside DMA into
          // LDS the compiler waits for every read there is, so here for this quarter's
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[0][j] = Elem<TY>::mma32(o.b[j], o.a[0], acc[0][j]);
          __builtin_amdgcn_sched_barrier(0);
          if (s < 3) {
            read(ops[(s + 1) & 1], st, s + 1);
          } else {
            // own reads of this stage done, own DMA of the next one landed, everyone
            // there: the next stage may be read and this one refilled
            wait_vm_barrier<0>();
            if constexpr (decltype(TAIL)::value) {
              if (after.rows) dma(kb + 2 - KB, stage);
            } else {
              dma(kb + 2, stage);
            }
            read(ops[0], nx, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 1; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = Elem<TY>::mma32(o.b[j], o.a[i], acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
        }
        stage ^= 1;
      };
      for (int kb = 0; kb + 2 < KB; ++kb) step(kb, std::false_type{});
      after = next();
      if (after.rows) sources(after);
      for (int kb = KB - 2; kb < KB; ++kb) step(kb, std::true_type{});
      uint8_t* turn = smem + 2 * kStage + wave * kTurn;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          store_block(p, turn, acc[i][j], cur.row0 + wm * 128 + i * 32, cur.rows - (wm * 128 + i * 32),
                      cur.nb0 + wn * 4 + j * 2);
      if (!after.rows) break;
      cur = after;
    }
  }
};

// Dense: one workgroup a CU; XCD x (workgroups b with b % 8 == x) walks over its own
// contiguous eighth of the tiles, 8 rows of tiles at a time, so that the tiles it
// runs together share panels in its L2.
template <int TY>
__global__ __launch_bounds__(512) void fused_wide_kernel(FusedGemm p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[WideTile<TY>::kLdsBytes];
  const int64_t MT = (p.M + 255) / 256, NT = (p.NB + 15) / 16, total = MT * NT;
  const int64_t per = (total + 7) / 8, first = (blockIdx.x % 8) * per, end = min(first + per, total);
  int64_t t = first + blockIdx.x / 8;
  WideTile<TY>::run(p, smem, [&]() __attribute__((always_inline)) {
    typename WideTile<TY>::Where w{0, 0, 0};
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

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// (offsets within a tile's 256 rows have 32 bits)
bool fused_rows_ok(const FusedGemm& p) {
  return p.lda % 16 == 0 && p.lda < (int64_t)1 << 24 && p.kbytes % 16 == 0 && ((uintptr_t)p.a & 15) == 0;
}

enum FusedKernel { kDecode16, kDecode16x32, kDecode32, kDecode64, kTile32, kTile64, kTile128, kTile256 };

static FusedKernel fused_kernel(const FusedGemm& p) {
  if (p.M > 1024 && p.KP > 2) return kTile256;  // its pipeline is two steps deep
  if (p.M > 64) return kTile128;
  if (p.M > 32) return kDecode64;
  if (p.M > 16) return kDecode32;
  return p.act == W8A8_ACT_SWIGLU ? kDecode16x32 : kDecode16;
}

bool fused_needs_copy(const FusedGemm& p) {
  return p.kbytes < 16 || (fused_kernel(p) == kTile256 && !fused_rows_ok(p));
}

int64_t fused_copy_bytes(int64_t M, int64_t kbytes) { return round_up(kbytes, kStepBytes) * M; }

// U: a wavefront's steps of K, at most as many as registers hold (sets without a step of
// their own load the last one again)
template <int TY, int MB, int NBW>
static void launch_decode(const FusedGemm& p, hipStream_t stream) {
  constexpr int kMost = MB * NBW >= 8 ? 2 : MB * NBW >= 4 ? 4 : 8;
  const int64_t steps = ceil_div(ceil_div(p.KP, 2), kDecodeWaves);
  auto fn = steps <= 2 ? fused_decode_kernel<TY, MB, NBW, 2>
          : steps <= 4 ? fused_decode_kernel<TY, MB, NBW, std::min(4, kMost)> : fused_decode_kernel<TY, MB, NBW, kMost>;
  hipLaunchKernelGGL(fn, dim3((unsigned)ceil_div(p.NB, NBW), (unsigned)ceil_div(p.M, 16 * MB)), dim3(kDecodeWaves * 64),
                     0, stream, p);
}

template <int TY, int MB, int NBW>
static void launch_tiles(const FusedGemm& p, hipStream_t stream) {
  hipLaunchKernelGGL((fused_dense_kernel<TY, MB, NBW>),
                     dim3((unsigned)ceil_div(p.M, MB * 16), (unsigned)ceil_div(p.NB, 8 * NBW)), dim3(512), 0, stream, p);
}

template <int TY>
static hipError_t launch_dense(const FusedGemm& p, FusedKernel kernel, hipStream_t stream) {
  switch (kernel) {
    case kDecode16: launch_decode<TY, 1, 1>(p, stream); break;
    case kDecode16x32: launch_decode<TY, 1, 2>(p, stream); break;
    case kDecode32: launch_decode<TY, 2, 2>(p, stream); break;
    case kDecode64: launch_decode<TY, 4, 2>(p, stream); break;
    case kTile32: launch_tiles<TY, 2, 2>(p, stream); break;
    case kTile64: launch_tiles<TY, 4, 2>(p, stream); break;
    case kTile128: launch_tiles<TY, 8, 2>(p, stream); break;
    case kTile256: {
      const int64_t tiles = ceil_div(p.M, 256) * ceil_div(p.NB, 16);
      hipLaunchKernelGGL(fused_wide_kernel<TY>, dim3((unsigned)std::min<int64_t>(256, round_up(tiles, 8))), dim3(512), 0,
                         stream, p);
      break;
    }
  }
  return hipGetLastError();
}

hipError_t launch_fused_gemm(FusedGemm p, void* room, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  if (p.group_list) {
    const int64_t NT = grouped_columns(p.NB * 16);
    hipLaunchKernelGGL((fused_grouped_kernel<kFusedBf16, kGroupedNBW>), dim3((unsigned)fused_grid(p.M, p.E, p.NB * 16)),
                       dim3(512), 0, stream, p, (int)NT);
    return hipGetLastError();
  }
  const FusedKernel kernel = fused_kernel(p);
  if (fused_needs_copy(p)) {
    const int64_t per = round_up(p.kbytes, kStepBytes) / 16;
    hipLaunchKernelGGL(fused_copy_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(p.M * per, 256), 1 << 16)), dim3(256),
                       0, stream, p.a, p.M, p.lda, p.kbytes, per, reinterpret_cast<uint8_t*>(room));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    p.a = reinterpret_cast<const uint8_t*>(room);
    p.lda = p.kbytes = per * 16;
  }
  return p.type == kFusedInt8 ? launch_dense<kFusedInt8>(p, kernel, stream) : launch_dense<kFusedBf16>(p, kernel, stream);
}

}  // namespace w8a8
