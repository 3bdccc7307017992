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

__device__ __forceinline__ int64_t outputs_of(const FusedGemm& p) { return p.act == W8A8_ACT_SWIGLU ? p.N / 2 : p.N; }

// A lane's four neighbouring output columns c .. c + 3: what belongs to them and not to a
// row, loaded once for all the rows of a tile. WHOLE: the columns exist, for every lane
// of the wavefront (a path of its own: with a choice at every access the epilogue of a
// 128 x 256 tile took 8 us).
struct Cols {
  int c;
  int n;  // of the four that exist; 0: none
  float bias[4], second[4];  // second: INT8 the columns' scales, SwiGLU the up half's bias
};

template <int TY, bool WHOLE>
__device__ __forceinline__ Cols load_cols(const FusedGemm& p, int64_t c) {
  const int64_t width = outputs_of(p);
  const bool swiglu = TY == kFusedBf16 && p.act == W8A8_ACT_SWIGLU;
  Cols o;
  o.c = (int)c;
  o.n = WHOLE ? 4 : (int)max((int64_t)0, min((int64_t)4, width - c));
  Bytes8 b{{kNothing2, kNothing2}}, u = b;
  Floats4 f{};
  if (p.bias) b = load_raw4<WHOLE>(p.bias + c, o.n);
  if (swiglu && p.bias) u = load_raw4<WHOLE>(p.bias + width + c, o.n);
  if (TY == kFusedInt8) {
    if (WHOLE) {
      f = *reinterpret_cast<const Floats4*>(p.w_scale + c);
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t < o.n) f.v[t] = p.w_scale[c + t];
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    o.bias[t] = bf16_of(b, t);
    o.second[t] = TY == kFusedInt8 ? f.v[t] : bf16_of(u, t);
  }
  return o;
}

// Takes the columns' values here: their loads are waited for now and not in a loop that
// stores, where each such wait is one for the stores too (loads and stores count as one;
// 0.9 us for every 16 rows).
__device__ __forceinline__ void arrived(Cols& o) {
#pragma unroll
  for (int t = 0; t < 4; ++t) asm volatile("" : "+v"(o.bias[t]), "+v"(o.second[t]));
}

// the residual of row m at the lane's columns, as it lies in memory
template <bool WHOLE>
__device__ __forceinline__ Bytes8 load_residual(const FusedGemm& p, int64_t m, const Cols& o) {
  return load_raw4<WHOLE>(p.residual + m * p.ldr + o.c, o.n);
}

// The outputs of row m from the sums of its four weight rows (SwiGLU: and of their
// partners `up`).
// ACT: p.act, or kAnyAct
template <int TY, bool WHOLE, int ACT, class Acc>
__device__ __forceinline__ void emit4(const FusedGemm& p, int64_t m, const Cols& o, float xs, const Bytes8& res,
                                      const Acc& acc, const Acc& up) {
  float v[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) v[t] = scaled(p, acc[t], xs, o.second[t]) + o.bias[t];
  const int act = ACT == kAnyAct ? p.act : ACT;
  if (TY == kFusedBf16 && act == W8A8_ACT_SWIGLU) {
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = times_sigmoid(v[t], v[t]) * ((float)up[t] + o.second[t]);
  } else {
    activate4(act, v);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) v[t] = v[t] + bf16_of(res, t);
  if (p.f32) {
    float* y = reinterpret_cast<float*>(p.y) + m * p.ldy + o.c;
    if (WHOLE) {
      *reinterpret_cast<Floats4*>(y) = Floats4{{v[0], v[1], v[2], v[3]}};
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t < o.n) y[t] = v[t];
    }
  } else {
    uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + m * p.ldy + o.c;
    uint32_t q[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) q[t] = to_bf16(v[t]);
    if (WHOLE) {
      *reinterpret_cast<Bytes8*>(y) = Bytes8{{q[0] | (q[1] << 16), q[2] | (q[3] << 16)}};
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t < o.n) y[t] = (uint16_t)q[t];
    }
  }
}

// first output column of the 16 x 16 blocks from nb on (SwiGLU: nb even)
__device__ __forceinline__ int64_t first_col(const FusedGemm& p, int64_t nb) {
  return (p.act == W8A8_ACT_SWIGLU ? nb / 2 : nb) * 16;
}

// The 16 x 16 block nb of weight rows against the rows of m: this lane's four outputs.
template <int TY, bool WHOLE, class Acc>
__device__ __forceinline__ void emit_one(const FusedGemm& p, int64_t m, int64_t c, const Acc& acc, const Acc& up) {
  const Cols o = load_cols<TY, WHOLE>(p, c);
  Bytes8 res{{kNothing2, kNothing2}};
  if (p.residual) res = load_residual<WHOLE>(p, m, o);
  emit4<TY, WHOLE, kAnyAct>(p, m, o, row_scale<TY>(p, m), res, acc, up);
}
template <int TY, class Acc>
__device__ __forceinline__ void emit_block(const FusedGemm& p, int64_t m, int64_t nb, int lane, const Acc& acc,
                                           const Acc& up) {
  const int64_t c0 = first_col(p, nb), c = c0 + (lane >> 4) * 4;
  if (c0 + 16 <= outputs_of(p)) emit_one<TY, true>(p, m, c, acc, up);  // wave-uniform
  else emit_one<TY, false>(p, m, c, acc, up);
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
// rows, 0} for every tile: in expert order the wide tiles of at most 256 rows of one
// expert, while more than kTileRows are left, then (what takes longest starts first) the
// tiles of at most tile_rows.
// ---------------------------------------------------------------------------
constexpr int kTileRows = 128, kWideRows = 256;

static int64_t max_tiles(int64_t R, int64_t E, int tile_rows) { return R / tile_rows + std::min(R, E); }

// one workgroup of 256 threads, four experts each (E <= 1024)
__global__ __launch_bounds__(256) void fused_schedule_kernel(const int64_t* __restrict__ group_list, int E, int64_t R,
                                                             int wide, int tile_rows, int* count, int4* tiles) {
  __shared__ int64_t wrows[4];
  __shared__ int64_t wtiles[4];
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
  // tiles, wide ones in the upper half
  int64_t row0[4], t = 0;
  auto wide_tiles = [&](int64_t rows) { return wide ? rows / kWideRows + (rows % kWideRows > kTileRows) : 0; };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    row0[i] = min(ri, R);
    ri += n[i];
    n[i] = min(n[i], R - row0[i]);
    const int64_t full = wide_tiles(n[i]), left = max(n[i] - full * kWideRows, (int64_t)0);
    t += (full << 32) + (left + tile_rows - 1) / tile_rows;
  }
  int64_t ti = t;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(ti, d, 64);
    if (lane >= d) ti += o;
  }
  if (lane == 63) wtiles[wave] = ti;
  __syncthreads();
  int64_t all = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) ti += wtiles[w];
    all += wtiles[w];
  }
  const int wides = (int)(all >> 32);
  if (tid == 0) *count = wides + (int)all;
  ti -= t;
  int at = (int)(ti >> 32), low = wides + (int)ti;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int64_t r = 0;
    for (int64_t k = wide_tiles(n[i]); k; --k, r += kWideRows)
      tiles[at++] = int4{4 * tid + i, (int)(row0[i] + r), (int)min(n[i] - r, (int64_t)kWideRows), 0};
    for (; r < n[i]; r += tile_rows)
      tiles[low++] = int4{4 * tid + i, (int)(row0[i] + r), (int)min(n[i] - r, (int64_t)tile_rows), 0};
  }
}

// Place of 16-byte chunk c (0..7) of row r (0..15) of a 16 x 128-byte block in LDS, for
// rows loaded as whole lines (a load whose neighbouring lanes lie in different rows costs
// the L1 a look-up for every 16 bytes, this one for every 128: tiles of 64 x 128 took 0.39
// us a step) and read as operands, 16 rows of one chunk: both ways 16 lanes meet all 64
// banks.
__device__ __forceinline__ uint32_t turned(int r, int c) {
  return (c >> 2) * kPiece + (c & 3) * 256 + ((r ^ (2 * c)) & 15) * 16;
}

// ---------------------------------------------------------------------------
// Streaming tile: up to 16 MB rows x 128 NBW columns over the whole K, eight
// wavefronts. Wavefront w owns the NBW 16-column blocks nb0 + NBW w + j and takes their
// weights from global memory straight into operand registers, kAhead steps ahead: every
// weight byte of the tile is read once and never passes through LDS. The rows, which
// all eight share, go through LDS one step at a time (four buffers, one barrier a step).
// Bound by what the L2 hands a CU, 32 bytes a clock: 64 x 128 take 24 KB a step, 0.32 us
// (at 128 x 256 48 KB and 0.81 us, of which the MFMAs are 0.43). 1024 x 4096 x 4096 in
// BF16: 64 x 128 49.8 us, 64 x 256 45.6, 128 x 256 59.7.
// ---------------------------------------------------------------------------
template <int TY, int MB, int NBW>
struct StreamTile {
  using Acc = typename Elem<TY>::Acc4;
  static constexpr int kSets = 4, kAhead = kSets - 1;          // steps of weights in flight
  static constexpr int kWaves = 8;
  static constexpr int kPieces = (2 * MB + kWaves - 1) / kWaves;  // 16-byte pieces a thread stages per step
  static constexpr int kBufBytes = MB * 2 * kPiece;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kSumBytes = MB * 16 * 128 * NBW * 4;
  static constexpr int kStoreBytes = kSumBytes + MB * 16 * 4;  // sums, row scales
  static constexpr int kLdsBytes = 4 * kBufBytes > kStoreBytes ? 4 * kBufBytes : kStoreBytes;

  struct Stage {
    i32x4 a[kPieces];
  };
  struct Weights {
    i32x4 v[NBW][2];
  };

  // Steps [k0, k1) of K. part: the sums go there as they are (a tile's kPartBytes, one 16 x
  // 16 block after the other), for the join of a product whose K is split.
  static constexpr int64_t kPartBytes = (int64_t)kWaves * MB * NBW * kPiece;

  __device__ __forceinline__ static void run(const FusedGemm& p, uint8_t* smem, int e, int64_t row0, int rows, int nb0,
                                             int k0, int k1, uint8_t* part) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int NB = (int)p.NB, KP = (int)p.KP, KB = (KP + 1) / 2;
    const uint32_t last = (uint32_t)p.kbytes - 16;
    const int nbw = nb0 + wave * NBW;
    // This thread's pieces of a step: 8 rows x 128 bytes (whole cache lines) each, piece
    // wave + 8 i, lane: row l / 8, 16-byte chunk l % 8. Rows past the tile read its last
    // row; they only feed outputs that are never stored.
    const uint8_t* ap[kPieces];
    const uint32_t at = (lane & 7) * 16;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = min((wave + kWaves * i) * 8 + (lane >> 3), rows - 1);
      int64_t src = row0 + r;
      if (p.row_index) src = max((int64_t)0, min((int64_t)p.row_index[src], p.a_rows - 1));
      ap[i] = p.a + src * p.lda;
    }
    const uint8_t* wp[NBW];
#pragma unroll
    for (int j = 0; j < NBW; ++j)  // blocks past the last read it; their outputs are never stored
      wp[j] = p.w + ((int64_t)e * NB + min(nbw + j, NB - 1)) * KP * kPiece;
    const uint32_t l16 = lane * 16;

    auto load_w = [&](Weights& w, int kb) __attribute__((always_inline)) {
      // an odd last piece is read twice: a is zero there
      kb = min(kb, k1 - 1);
      const int64_t c0 = 2 * kb, c1 = min(2 * kb + 1, KP - 1);
#pragma unroll
      for (int j = 0; j < NBW; ++j) {
        w.v[j][0] = *reinterpret_cast<const i32x4*>(wp[j] + c0 * kPiece + l16);
        w.v[j][1] = *reinterpret_cast<const i32x4*>(wp[j] + c1 * kPiece + l16);
      }
    };
    auto load_a = [&](Stage& st, int kb) __attribute__((always_inline)) {
      const uint32_t k = (uint32_t)min(kb, k1 - 1) * kStepBytes;
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (2 * MB >= kWaves * (i + 1) || wave + kWaves * i < 2 * MB) st.a[i] = load16(ap[i], k + at, last);
    };
    auto store_a = [&](Stage& st, uint8_t* buf, int kb) __attribute__((always_inline)) {
      if (min(kb, k1 - 1) == KB - 1) {  // the last step (or a copy of it)
        const int past = (KB - 1) * kStepBytes - (int)last + (int)at;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) st.a[i] = fix16(st.a[i], past);
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int piece = wave + kWaves * i;
        if (2 * MB >= kWaves * (i + 1) || piece < 2 * MB)
          *reinterpret_cast<i32x4*>(buf + (piece >> 1) * 2 * kPiece + turned((piece & 1) * 8 + (lane >> 3), lane & 7)) =
              st.a[i];
      }
    };

    Acc acc[MB][NBW];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int j = 0; j < NBW; ++j) acc[m][j] = Acc{0, 0, 0, 0};

    constexpr int kD = MB * NBW > 2 ? 2 : MB, kF = 2 * kD;
    struct Frag {
      i32x4 v[2];
    };
    Frag f[kF];
    const uint32_t r0 = turned(lane & 15, lane >> 4);  // the second half's chunks: 4 more, so ^ 128
    auto read_a = [&](Frag& d, const uint8_t* buf, int m) __attribute__((always_inline)) {
      d.v[0] = *reinterpret_cast<const i32x4*>(buf + m * 2 * kPiece + r0);
      d.v[1] = *reinterpret_cast<const i32x4*>(buf + m * 2 * kPiece + (r0 ^ 128) + kPiece);
    };
    // Step kb: weights in set (kb - k0) % 4, rows in that buffer. The weights of kb + 3 and
    // the rows of kb + 5 are loaded; kb is multiplied, each operand read kD row blocks
    // before its MFMAs (the first ones in the step before, so that no wavefront waits for
    // LDS right behind the barrier); the rows of kb + 2, loaded three steps ago, go to their
    // buffer, last read in step kb - 2, and are read from the end of step kb + 1 on, behind
    // the barrier of step kb. Loads past the last step read it again.
    Weights w[kSets];
    Stage st[4];  // rows of step d in st[(d - k0 - 2) % 4]
    {
      // the order of the steps before k0, so that the waits of the loop fit its start too
      Stage first[2];
      load_a(first[0], k0);
      load_a(first[1], k0 + 1);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        load_a(st[i], k0 + 2 + i);
        load_w(w[i], k0 + i);
      }
      store_a(first[0], smem, k0);
      store_a(first[1], smem + kBufBytes, k0 + 1);
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < kD; ++i) read_a(f[i], smem, i);
    auto step = [&](int kb, auto STEP) __attribute__((always_inline)) {
      constexpr int I = decltype(STEP)::value;
      const uint8_t* buf = smem + I % 4 * kBufBytes;
      const uint8_t* next = smem + ((I + 1) % 4) * kBufBytes;
      load_a(st[(I + 3) & 3], kb + 5);
      load_w(w[(I + kAhead) % kSets], kb + kAhead);
      const auto& wk = w[I].v;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        read_a(f[(I * MB + m + kD) % kF], m + kD < MB ? buf : next, (m + kD) % MB);
        __builtin_amdgcn_sched_barrier(0);
        const Frag& a = f[(I * MB + m) % kF];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int j = 0; j < NBW; ++j) acc[m][j] = Elem<TY>::mma16(wk[j][q], a.v[q], acc[m][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      store_a(st[I & 3], smem + ((I + 2) % 4) * kBufBytes, kb + 2);
      lds_barrier();
    };
    // Whole rounds of the register sets without an exit between, then the rest in a line
    // of its own: an exit inside the round, though it only leaves the loop, makes the
    // compiler's waits at its head drain the loads in flight
    int kb = k0;
#pragma unroll 1
    for (; kb + kSets <= k1; kb += kSets) {
      step(kb, std::integral_constant<int, 0>{});
      step(kb + 1, std::integral_constant<int, 1>{});
      step(kb + 2, std::integral_constant<int, 2>{});
      step(kb + 3, std::integral_constant<int, 3>{});
    }
    if (kb < k1) {
      step(kb, std::integral_constant<int, 0>{});
      if (kb + 1 < k1) {
        step(kb + 1, std::integral_constant<int, 1>{});
        if (kb + 2 < k1) step(kb + 2, std::integral_constant<int, 2>{});
      }
    }
    if (part) {
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < NBW; ++j)
          *reinterpret_cast<Acc*>(part + ((wave * MB + m) * NBW + j) * kPiece + l16) = acc[m][j];
      return;
    }
    int et = threadIdx.x;
    asm volatile("" : "+v"(et));  // read here, not kept over the K loop
    const int64_t c0 = first_col(p, nb0), width = outputs_of(p);
    if (c0 + (p.act == W8A8_ACT_SWIGLU ? 64 * NBW : 128 * NBW) <= width) store_tile<true>(p, smem, acc, row0, rows, c0, et);
    else store_tile<false>(p, smem, acc, row0, rows, c0, et);
  }

  // The sums through LDS, from where the wavefronts store whole rows of the tile in a loop
  // of few branches (unrolled, with the choices at every output, the epilogue of a 128 x 256
  // tile was 65 KB of code; 4096 x 4096 x 64 took 22.0 us in tiles of 64 x 128, now 17.6).
  template <bool WHOLE>
  __device__ __forceinline__ static void store_tile(const FusedGemm& p, uint8_t* smem, const Acc (&acc)[MB][NBW],
                                                    int64_t row0, int rows, int64_t c0, int tid) {
    const int shift = p.act == W8A8_ACT_SWIGLU ? kTurnShift - 1 : kTurnShift;  // log2 of a row's lanes
    const int c4 = tid & ((1 << shift) - 1);
    float* scales = reinterpret_cast<float*>(smem + kSumBytes);
    float xs = 0.0f;
    if (TY == kFusedInt8) xs = row_scale<TY>(p, row0 + min(tid, rows - 1));
    Cols cols = load_cols<TY, WHOLE>(p, c0 + c4 * 4);
    lds_barrier();  // every wavefront is done with its operands
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int j = 0; j < NBW; ++j)
        *reinterpret_cast<Acc*>(smem + sums_at(m * 16 + (tid & 15), ((tid >> 6) * NBW + j) * 4 + ((tid >> 4) & 3))) =
            acc[m][j];
    if (TY == kFusedInt8 && tid < MB * 16) scales[tid] = xs;
    lds_barrier();
    arrived(cols);
    if constexpr (WHOLE) {
      for_act<TY == kFusedBf16>(p.act, [&](auto ACT) __attribute__((always_inline)) {
        store_rows<WHOLE, decltype(ACT)::value>(p, smem, scales, cols, row0, rows, tid);
      });
    } else {
      store_rows<WHOLE, kAnyAct>(p, smem, scales, cols, row0, rows, tid);
    }
  }

  template <bool WHOLE, int ACT>
  __device__ __forceinline__ static void store_rows(const FusedGemm& p, const uint8_t* smem, const float* scales,
                                                    const Cols& cols, int64_t row0, int rows, int tid) {
    const bool swiglu = ACT == kAnyAct ? p.act == W8A8_ACT_SWIGLU : ACT == W8A8_ACT_SWIGLU;
    const int shift = swiglu ? kTurnShift - 1 : kTurnShift;
    const int c4 = tid & ((1 << shift) - 1);
    const int chunk = swiglu ? (c4 >> 2) * 8 + (c4 & 3) : c4;  // 16 gate columns, then their 16 up columns
    constexpr int kRows = 4;  // of a lane at a time, their residual together
#pragma unroll 1
    for (int r0 = tid >> shift; r0 < rows; r0 += kRows * kThreads >> shift) {
      Bytes8 res[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) res[k] = Bytes8{{kNothing2, kNothing2}};
      if (p.residual) {
#pragma unroll
        for (int k = 0; k < kRows; ++k)
          res[k] = load_residual<WHOLE>(p, row0 + min(r0 + (k * kThreads >> shift), rows - 1), cols);
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int r = r0 + (k * kThreads >> shift);
        if (r < rows) {
          const Acc v = *reinterpret_cast<const Acc*>(smem + sums_at(r, chunk));
          const Acc up = *reinterpret_cast<const Acc*>(smem + sums_at(r, chunk ^ 4));
          emit4<TY, WHOLE, ACT>(p, row0 + r, cols, TY == kFusedInt8 ? scales[r] : 0.0f, res[k], v, up);
        }
      }
    }
  }

  // Sums on their way to whole rows: rows of 128 NBW columns, 16-byte chunk c of row r in
  // slot c ^ r % 16, so that a column's 16 chunks lie in all 64 banks.
  static constexpr int kTurnShift = NBW == 2 ? 6 : 5;  // log2 of the 16-byte chunks of a row
  __device__ __forceinline__ static int sums_at(int r, int c) { return (r << (kTurnShift + 4)) + ((c ^ (r & 15)) << 4); }
};

// Dense: tiles of one height. S > 1: K in S parts of `per` steps each, whose sums
// fused_join_kernel adds. Workgroup b runs on XCD b % 8: each XCD takes its own
// contiguous eighth of the tiles, rows first, so that its L2 reads the weights of its
// columns once (BF16 195 x 4684 x 4720, 32-row tiles: 60.7 us in launch order, here 35.7;
// 1024 x 4096 x 4096, 64 x 256 tiles: 56.2, 45.6; 4096 x 512 x 2048, 64-row tiles: 15.1,
// 16.2).
template <int TY, int MB, int NBW>
__global__ __launch_bounds__(512) void fused_dense_kernel(FusedGemm p, int S, int per, uint8_t* part) {
  using T = StreamTile<TY, MB, NBW>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::kLdsBytes];
  uint32_t bx = blockIdx.x, by = blockIdx.y, bz = blockIdx.z;
  const uint64_t total = (uint64_t)gridDim.x * gridDim.y * gridDim.z;
  if (total < (uint64_t)1 << 31) {
    const uint32_t b = bx + gridDim.x * (by + gridDim.y * bz), n = (uint32_t)total;
    const uint32_t t = b % 8 * (n / 8) + min(b % 8, n % 8) + b / 8;
    bx = t % gridDim.x;
    by = t / gridDim.x % gridDim.y;
    bz = t / gridDim.x / gridDim.y;
  }
  const int64_t row0 = (int64_t)bx * (MB * 16);
  const int KB = (int)(p.KP + 1) / 2, k0 = bz * per;
  uint8_t* mine = nullptr;
  if (S > 1) mine = part + (((int64_t)bz * gridDim.y + by) * gridDim.x + bx) * T::kPartBytes;
  T::run(p, smem, 0, row0, (int)min((int64_t)(MB * 16), p.M - row0), by * 8 * NBW, k0, min(KB, k0 + per), mine);
}

// The S parts of every 16 x 16 block, in their order, and the epilogue: a wavefront a
// block (SwiGLU: a pair of blocks).
template <int TY, int MB, int NBW>
__global__ __launch_bounds__(256) void fused_join_kernel(FusedGemm p, int S, int rows_of_tiles, int64_t tiles,
                                                         const uint8_t* part) {
  using Acc = typename Elem<TY>::Acc4;
  constexpr int kBlocks = 8 * MB * NBW;  // of a tile
  const int lane = threadIdx.x & 63;
  const int64_t b = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t tile = b / kBlocks;
  if (tile >= tiles) return;
  const int at = (int)(b % kBlocks), wave = at / (MB * NBW), m = at / NBW % MB, j = at % NBW;
  const int64_t nb = tile / rows_of_tiles * (8 * NBW) + wave * NBW + j;
  const int64_t r = tile % rows_of_tiles * (MB * 16) + m * 16 + (lane & 15);
  const bool swiglu = p.act == W8A8_ACT_SWIGLU;
  if ((swiglu && (nb & 1)) || nb >= p.NB) return;
  auto total = [&](int64_t off) __attribute__((always_inline)) {
    const uint8_t* src = part + tile * kBlocks * kPiece + off * kPiece + lane * 16;
    Acc sum = *reinterpret_cast<const Acc*>(src);
#pragma unroll 8
    for (int s = 1; s < S; ++s) sum += *reinterpret_cast<const Acc*>(src + s * tiles * kBlocks * kPiece);
    return sum;
  };
  const Acc sum = total(at);
  // the up block: the next of this wavefront's, or the next wavefront's
  if (swiglu) {
    const Acc up = total(NBW == 1 ? at + MB : at + 1);
    if (r < p.M) emit_block<TY>(p, r, nb, lane, sum, up);
  } else if (r < p.M) {
    emit_block<TY>(p, r, nb, lane, sum, sum);
  }
}

// ---------------------------------------------------------------------------
// Decode (dense, few rows): the weight's stream, split over K inside the workgroup. A
// workgroup owns NBW 16-column blocks and 16 MB rows over the whole K; its eight
// wavefronts take every eighth step, with U steps of weights and rows in flight each,
// straight from global memory into operand registers and each set refilled as soon as
// it is multiplied, and their sums meet in LDS in a fixed order. Bound by the weights'
// stream (BF16 1 x 4096 x 7168: 12.7 us with the weights in HBM, 4.6 TB/s; 9.2 to 10.5 with
// them in the memory-side cache) and with tens of rows by what the L2 hands a CU, 32 bytes a
// clock (256 x 256 x 7168: 4 KB a step, 458 KB a CU, 8.0 us; INT8 64 x 4096 x 7168: as much in
// tiles of 32 x 32, 11.6 from HBM).
// ---------------------------------------------------------------------------
constexpr int kDecodeWaves = 8;

template <int TY, int MB, int NBW, int U>
__global__ __launch_bounds__(kDecodeWaves * 64) void fused_decode_kernel(FusedGemm p) {
  using Acc = typename Elem<TY>::Acc4;
  // a wavefront's rows on their way into operand order, two steps; then the sums
  constexpr int kTurn = 2 * MB * 2 * kPiece, kRed = MB * NBW * kPiece;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kDecodeWaves * (kTurn > kRed ? kTurn : kRed)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int NB = (int)p.NB, KP = (int)p.KP, KB = (KP + 1) / 2, M = (int)p.M;
  const uint32_t last = (uint32_t)p.kbytes - 16;
  const int nb0 = blockIdx.x * NBW, m0 = blockIdx.y * MB * 16;
  const uint32_t l16 = lane * 16, at = (lane & 7) * 16;
  const uint8_t* wp[NBW];
#pragma unroll
  for (int j = 0; j < NBW; ++j)  // blocks past the last read it; their outputs are never stored
    wp[j] = p.w + (int64_t)min(nb0 + j, NB - 1) * KP * kPiece;
  const uint8_t* ap[MB][2];  // rows past the last read it; they only feed outputs that are never stored
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) ap[m][h] = p.a + (int64_t)min(m0 + m * 16 + h * 8 + (lane >> 3), M - 1) * p.lda;

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
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) a[u][m][h] = load16(ap[m][h], k, last);
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
  uint8_t* const mine = smem + wave * kTurn;
  const uint32_t to0 = turned(lane >> 3, lane & 7), to1 = turned(8 + (lane >> 3), lane & 7);
  const uint32_t from = turned(lane & 15, lane >> 4);
  // the rows of set u, step kb (this wavefront's n-th), into LDS: one step ahead of its product
  auto turn = [&](int u, int kb, int n) __attribute__((always_inline)) {
    uint8_t* buf = mine + (n & 1) * MB * 2 * kPiece;
    if (kb == KB - 1) {  // wave-uniform
      const int past = (KB - 1) * kStepBytes - (int)last + (int)at;
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) a[u][m][h] = fix16(a[u][m][h], past);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      *reinterpret_cast<i32x4*>(buf + m * 2 * kPiece + to0) = a[u][m][0];
      *reinterpret_cast<i32x4*>(buf + m * 2 * kPiece + to1) = a[u][m][1];
    }
  };
  auto mul = [&](int u, int n) __attribute__((always_inline)) {
    const uint8_t* buf = mine + (n & 1) * MB * 2 * kPiece;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const i32x4 x = *reinterpret_cast<const i32x4*>(buf + m * 2 * kPiece + q * kPiece + (q ? from ^ 128 : from));
#pragma unroll
        for (int j = 0; j < NBW; ++j) acc[m][j] = Elem<TY>::mma16(w[u][j][q], x, acc[m][j]);
      }
  };
  __builtin_amdgcn_sched_barrier(0);  // every first load in flight before the first product
  int kb0 = wave;
  static_assert(U % 2 == 0, "the two LDS buffers alternate over a round");
  turn(0, kb0, 0);
  for (; kb0 + kDecodeWaves * U < KB; kb0 += kDecodeWaves * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // set 0 again at the end: refilled in this round
      turn((u + 1) % U, kb0 + (u + 1) * kDecodeWaves, u + 1);
      mul(u, u);
      load_a(u, kb0 + (u + U) * kDecodeWaves);
      load_w(u, kb0 + (u + U) * kDecodeWaves);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (kb0 < KB) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb0 + u * kDecodeWaves >= KB) break;  // wave-uniform: clamped steps add nothing
      if (u + 1 < U) turn(u + 1, kb0 + (u + 1) * kDecodeWaves, u + 1);
      mul(u, u);
    }
  }
  __syncthreads();  // every wavefront is done with its rows
  auto red = reinterpret_cast<Acc(*)[MB * NBW][kWave]>(smem);
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
  const Acc sum = total(swiglu ? wave * 2 : wave);
  emit_block<TY>(p, r, nb0 + wave % per, lane, sum, swiglu ? total(wave * 2 + 1) : sum);
}

// ---------------------------------------------------------------------------
// Wide tiles: 256 rows x 256 columns over the whole K, eight wavefronts (2 x 4, each
// 128 x 64 as 4 x 2 blocks of the 32 x 32 MFMA), both operands through LDS by DMA.
//
// LDS: two stages of one step, each 32 pieces of 8 rows x 128 bytes of a (whole cache
// lines; 16-byte chunk c of row r in slot c ^ (r / 2 % 8), so that 16 rows of an operand
// lie in all 64 banks) and 32 pieces of packed weight; and 4 KB a
// wavefront through which the sums are turned into whole lines of y.
// Step kb, in four quarters of 32 bytes of K: the operands of a quarter are read while
// the one before is multiplied; before the last quarter's MFMAs "own DMA of kb + 1
// landed, own reads of kb done, s_barrier", then the rows of kb + 2 into the stage of
// kb, and its weights in the next step's first quarter (all eight copies at once: the
// queue of the vector memory holds up the wavefront's products, 395 us for BF16 8192 x
// 4096 x 7168 where this form takes 382; one a product: 406). A workgroup walks over its
// tiles without a gap: the last two steps of a tile load the first two of the next one,
// which land while the tile is stored.
// BF16 8192^3 850 us (1.29 PFLOP/s; the vendor library's bare product 803), INT8 8192 x
// 4096 x 7168 203 (2.37 POPS; 238). A copy of the kernel that only multiplies takes 669 of
// the 850 at the clock that the data's power leaves, one without its copies 746.
// ---------------------------------------------------------------------------
static __device__ __align__(16) uint8_t zeros16[16];

template <int TY, bool DENSE>
struct WideTile {
  using Acc = typename Elem<TY>::Acc16;
  static constexpr int kOperand = 32768;  // one operand of one stage
  static constexpr int kStage = 2 * kOperand;
  static constexpr int kTurn = 4096;      // a wavefront's room in the epilogue
  static constexpr int kLdsBytes = 2 * kStage + 8 * kTurn;

  struct Where {
    int rows, nb0;  // rows, first column block; rows 0: no tile
    int64_t row0;
    int e;          // expert
  };

  // 16 of a 32 x 32 block's rows (half h) into LDS, beside those of the block to its
  // right: rows of 64 columns, 16-byte chunk c of row r in slot c ^ r.
  __device__ __forceinline__ static void turn_block(uint8_t* turn, const Acc& acc, int j, int h, int lane) {
    if (((lane >> 4) & 1) == h) {
      uint8_t* mine = turn + (lane & 15) * 256;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        typename Elem<TY>::Acc4 v;
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = acc[4 * g + t];
        *reinterpret_cast<typename Elem<TY>::Acc4*>(mine + (((8 * j + 2 * g + (lane >> 5)) ^ (lane & 15)) * 16)) = v;
      }
    }
  }

  // One copy of the epilogue behind a choice of the rows' registers. A lane takes 4
  // neighbouring columns, 16 (SwiGLU: eight) lanes a row, so every fourth (eighth) row.
  // What it loads is there before it stores: row scales in two registers, the residual of
  // 32 rows at a time.
  template <bool WHOLE, bool RES, int ACT>
  __device__ __forceinline__ static void store_tile(const FusedGemm& p, uint8_t* turn, const Acc (&acc)[4][2], int64_t row0,
                                                    int rows, int64_t c0, int lane) {
    using Acc4 = typename Elem<TY>::Acc4;
    const bool swiglu = ACT == kAnyAct ? p.act == W8A8_ACT_SWIGLU : ACT == W8A8_ACT_SWIGLU;
    const int shift = swiglu ? 3 : 4;
    const int c4 = lane & ((1 << shift) - 1);
    const int c = swiglu ? (c4 >> 2) * 8 + (c4 & 3) : c4;  // 16 gate columns, then their 16 up columns
    Cols cols = load_cols<TY, WHOLE>(p, c0 + c4 * 4);
    float xs[2] = {0.0f, 0.0f};  // of rows lane and 64 + lane
    if (TY == kFusedInt8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) xs[h] = row_scale<TY>(p, row0 + min(h * 64 + lane, rows - 1));
    }
    arrived(cols);
#pragma unroll
    for (int h = 0; h < 2; ++h) asm volatile("" : "+v"(xs[h]));
    auto row_of = [&](int k) __attribute__((always_inline)) { return (lane >> shift) + (k * 64 >> shift); };
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
      if (rows <= h * 32) break;
      Bytes8 ahead[2][4];
      if (RES) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            ahead[i][k] = load_residual<WHOLE>(p, row0 + min(h * 32 + i * 16 + min(row_of(k), 15), rows - 1), cols);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) asm volatile("" : "+v"(ahead[i][k].w[0]), "+v"(ahead[i][k].w[1]));
      }
      const float scale = h > 1 ? xs[1] : xs[0];
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const int first = h * 32 + i * 16;
        if (rows <= first) break;
        Bytes8 res[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) res[k] = RES ? i ? ahead[1][k] : ahead[0][k] : Bytes8{{kNothing2, kNothing2}};
        // (the same wavefront writes and reads its LDS: in order, no barrier)
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int I = 0; I < 4; ++I)
          if (h == I) {
            asm volatile("");
            turn_block(turn, acc[I][0], 0, i & 1, lane);
            turn_block(turn, acc[I][1], 1, i & 1, lane);
          }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = row_of(k);
          const float row_xs = TY == kFusedInt8 ? __shfl(scale, (first + (r & 15)) & 63) : 0.0f;
          if (r < min(rows - first, 16)) {
            const Acc4 v = *reinterpret_cast<const Acc4*>(turn + r * 256 + ((c ^ r) * 16));
            const Acc4 up = *reinterpret_cast<const Acc4*>(turn + r * 256 + ((c ^ 4 ^ r) * 16));
            if (!WHOLE && p.residual) res[k] = load_residual<WHOLE>(p, row0 + first + r, cols);
            emit4<TY, WHOLE, ACT>(p, row0 + first + r, cols, row_xs, res[k], v, up);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }

  // next(): this workgroup's next tile. At least two steps of K.
  template <class Next>
  __device__ __forceinline__ static void run(const FusedGemm& p, uint8_t* smem, Next next) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int NB = (int)p.NB, KP = (int)p.KP, KB = (KP + 1) / 2;
    const uint32_t l16 = lane * 16;
    // a lane number that is read here, not kept (with what follows from it) over the K loop
    auto fresh_lane = [&]() __attribute__((always_inline)) {
      int v = threadIdx.x & 63;
      asm volatile("" : "+v"(v));
      return v;
    };
    // of even pieces; odd ones: ^ 64
    auto own_chunk = [&]() __attribute__((always_inline)) {
      const int sl = fresh_lane();
      return (uint32_t)((sl & 7) ^ (sl >> 4)) * 16;
    };
    const bool ragged = p.kbytes != (int64_t)KB * kStepBytes;
    const uint8_t* abase;    // the tile's first row
    uint32_t aoff[4];        // this wavefront's four pieces of a: bytes from abase
    const uint8_t* wp[2];    // its two weight blocks
    auto sources = [&](const Where& t) __attribute__((always_inline)) {
      const int sl = fresh_lane();
      const uint32_t chunk = own_chunk();
      // rows past the tile read its last
      abase = p.row_index ? p.a : p.a + t.row0 * p.lda;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int r = min((wave * 4 + i) * 8 + (sl >> 3), t.rows - 1);
        if (p.row_index) r = (int)max((int64_t)0, min((int64_t)p.row_index[t.row0 + r], p.a_rows - 1));
        aoff[i] = (uint32_t)r * (uint32_t)p.lda + (chunk ^ (i & 1) * 64);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)  // past the last block, that one (never stored)
        wp[j] = p.w + ((int64_t)t.e * NB + min(t.nb0 + wave * 2 + j, NB - 1)) * KP * kPiece;
    };
    // Addresses are a wave-uniform base and a 32-bit lane offset; the empty asm keeps
    // the compiler from hoisting their sums into register pairs.
    auto dma_a = [&](int k, int stage) __attribute__((always_inline)) {
      W8A8_LDS uint8_t* dst = (W8A8_LDS uint8_t*)smem + stage * kStage;
      const uint8_t* ab = abase + (int64_t)k * kStepBytes;
      if (ragged && k == KB - 1) {  // the same in every lane
        const uint32_t chunk = own_chunk();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = (int64_t)k * kStepBytes + (chunk ^ (i & 1) * 64) < p.kbytes;
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
    };
    auto dma_w = [&](int k, int stage) __attribute__((always_inline)) {
      W8A8_LDS uint8_t* dst = (W8A8_LDS uint8_t*)smem + stage * kStage;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t o = l16;
        asm volatile("" : "+v"(o));
        const uint8_t* wb = wp[j >> 1] + (int64_t)min(2 * k + (j & 1), KP - 1) * kPiece;
        __builtin_amdgcn_global_load_lds(wb + o, (W8A8_LDS void*)(dst + kOperand + (wave * 4 + j) * 1024), 16, 0, 0);
      }
    };
    // operands of quarter s: 32 rows (l % 32), 16 bytes at l / 32 of its 32
    const uint32_t ar = (wm * 128 + (lane & 31)) * 128, a7 = (lane >> 1) & 7;
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
    dma_a(0, 0);
    dma_w(0, 0);
    dma_a(1, 1);
    dma_w(1, 1);
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
      Where after{};
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
            // the weights of kb + 1, behind the rows that the step before asked for
            if (s == 0 && kb > 0) {
              if constexpr (decltype(TAIL)::value) {
                if (kb < KB - 1) dma_w(kb + 1, stage ^ 1);
                else if (after.rows) dma_w(0, stage ^ 1);
              } else {
                dma_w(kb + 1, stage ^ 1);
              }
            }
            if constexpr (decltype(TAIL)::value) {
              if (s == 1 && kb == KB - 2) {  // every copy of this tile is on its way
                after = next();
                if (after.rows) sources(after);
              }
            }
          } else {
            // own reads of this stage done, own DMA of the next one landed, everyone
            // there: the next stage may be read and this one refilled
            wait_vm_barrier<0>();
            if constexpr (decltype(TAIL)::value) {
              if (kb < KB - 1) read(ops[0], nx, 0);  // the next tile's first: behind the epilogue
            } else {
              read(ops[0], nx, 0);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 1; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = Elem<TY>::mma32(o.b[j], o.a[i], acc[i][j]);
            if (s == 3 && i == 1) {
              __builtin_amdgcn_sched_barrier(0);
              if constexpr (decltype(TAIL)::value) {
                if (after.rows) {
                  dma_a(kb + 2 - KB, stage);
                  if (kb == KB - 1) dma_w(1, stage);
                }
              } else {
                dma_a(kb + 2, stage);
              }
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        stage ^= 1;
      };
      for (int kb = 0; kb + 2 < KB; ++kb) step(kb, std::false_type{});
      for (int kb = KB - 2; kb < KB; ++kb) step(kb, std::true_type{});
      uint8_t* turn = smem + 2 * kStage + wave * kTurn;
      const int el = fresh_lane();
      const int64_t c0 = first_col(p, cur.nb0 + wn * 4);
      const int64_t row0 = cur.row0 + wm * 128;
      const int rows = cur.rows - wm * 128;
      if (c0 + (p.act == W8A8_ACT_SWIGLU ? 32 : 64) > outputs_of(p)) {
        store_tile<false, false, kAnyAct>(p, turn, acc, row0, rows, c0, el);
      } else if (DENSE && p.residual) {
        store_tile<true, true, kAnyAct>(p, turn, acc, row0, rows, c0, el);
      } else {
        for_act<TY == kFusedBf16>(p.act, [&](auto ACT) __attribute__((always_inline)) {
          store_tile<true, false, decltype(ACT)::value>(p, turn, acc, row0, rows, c0, el);
        });
      }
      if (!after.rows) break;
      cur = after;
      read(ops[0], smem + stage * kStage, 0);
    }
  }
};

// Dense: one workgroup a CU; XCD x (workgroups b with b % 8 == x) walks over its own
// contiguous eighth of the tiles, 8 rows of tiles at a time, so that the tiles it
// runs together share panels in its L2.
template <int TY>
__global__ __launch_bounds__(512) void fused_wide_kernel(FusedGemm p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[WideTile<TY, true>::kLdsBytes];
  const int64_t MT = (p.M + 255) / 256, NT = (p.NB + 15) / 16, total = MT * NT;
  const int64_t per = (total + 7) / 8, first = (blockIdx.x % 8) * per, end = min(first + per, total);
  int64_t t = first + blockIdx.x / 8;
  WideTile<TY, true>::run(p, smem, [&]() __attribute__((always_inline)) {
    typename WideTile<TY, true>::Where w{};
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

// Grouped: every row tile times NT column groups; workgroup b runs on XCD b % 8. A
// tile's column groups go to two XCDs (one if NT is odd), whose L2 they read the tile's
// rows through, 4 or 8 tiles at a time.
constexpr int kSpreadTiles = 64;

// NBW 2: tiles of 128 rows x 256 columns, and wide ones; NBW 1: 64 rows x 128 columns,
// for products that would not fill the chip with those. 128 rows over 256 experts of 4096 x
// 4096 524 us (the weights at 6.1 TB/s); 16384 rows over 64 such experts 726 (0.76
// PFLOP/s: experts' last rows in lower tiles, 3.2 GB past the L2s where 2.2 would do). Walking on
// from wide tile to wide tile, as the dense kernel does, gained nothing (749, 754).
template <int TY, int NBW>
__global__ __launch_bounds__(512) void fused_grouped_kernel(FusedGemm p, int NT) {
  using T = WideTile<TY, false>;
  static_assert(StreamTile<TY, 8, 2>::kLdsBytes <= T::kLdsBytes, "one LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NBW == 2 ? T::kLdsBytes : StreamTile<TY, 4, 1>::kLdsBytes];
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
  const int e = __builtin_amdgcn_readfirstlane(tile.x), row0 = __builtin_amdgcn_readfirstlane(tile.y);
  const int rows = __builtin_amdgcn_readfirstlane(tile.z), nb0 = c * 8 * NBW, KB = (int)(p.KP + 1) / 2;
  auto run = [&](auto MB) __attribute__((always_inline)) {
    StreamTile<TY, decltype(MB)::value, NBW>::run(p, smem, e, row0, rows, nb0, 0, KB, nullptr);
  };
  if (rows <= 16) {
    run(std::integral_constant<int, 1>{});
  } else if (rows <= 32) {
    run(std::integral_constant<int, 2>{});
  } else if (NBW == 1 || rows <= 64) {
    run(std::integral_constant<int, 4>{});
  } else if constexpr (NBW == 2) {
    if (rows <= 96) {
      run(std::integral_constant<int, 6>{});
    } else if (rows <= kTileRows) {
      run(std::integral_constant<int, 8>{});
    } else {
      int left = 1;
      T::run(p, smem, [&]() __attribute__((always_inline)) {
        typename T::Where w{};
        if (left-- > 0) w = typename T::Where{rows, nb0, row0, e};
        return w;
      });
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// (offsets within a tile's 256 rows have 32 bits)
bool fused_rows_ok(const FusedGemm& p) {
  return p.lda % 16 == 0 && p.lda < (int64_t)1 << 24 && p.kbytes % 16 == 0 && ((uintptr_t)p.a & 15) == 0;
}

enum FusedKernel { kDecode16, kDecode16x32, kDecode32, kDecode64, kTile32, kTile64, kTile64x256, kTile128, kTile256 };

// What a product takes with each kernel, in us, by a model fitted to measured products of
// either type, M 1 .. 8192, N 32 .. 16384, K 64 .. 16384. Over 6375 others the kernel it
// picks is 1.9 % slower in the mean than the best of them, in one of a hundred 1.3 times, at
// worst 1.9 times (2183 x 205 x 10144); it ranks the kernels, as a time it is 0.85 to 1.12 of
// the measured one for eight of ten:
//   launch + rounds * round + steps * max(first, filling * step) + (split) join + parts
// rounds: workgroups over twice the CUs (wide: whole turns of one workgroup a CU); steps:
// 128-byte steps of K a workgroup goes through; first: such a step where the chip is not
// full; filling: rounds, for the decode kernels three quarters of the way to whole turns of
// one workgroup a CU. INT8 and BF16 take the same time for the same bytes of K. A split of K is taken
// into as many parts as give the chip half a workgroup, one or two a CU.
struct FusedCost {
  int rows, cols;
  double launch, round, first, step, join, part;  // part: per MB of partial sums
};
constexpr FusedCost kCost[] = {
    {16, 16, 2.5, 0.706, 0.0407, 0.124, 0, 0},        {16, 32, 2.7, 1.05, 0.061, 0.196, 0, 0},
    {32, 32, 3.01, 1.73, 0.0356, 0.242, 0, 0},        {64, 32, 3.51, 4.25, 0.122, 0.326, 0, 0},
    {32, 128, 3.25, 1.9, 0.257, 0.589, 3.07, 0.437},  {64, 128, 4.04, 2.55, 0.322, 0.809, 2.9, 0.255},
    {64, 256, 5.09, 6.77, 0.517, 1.38, 0, 0},         {128, 256, 7.37, 11.9, 0.808, 2.19, 2.18, 0.0812},
    {256, 256, 3.36, 10.9, 1.23, 1.3, 0, 0},
};

static double tiles_time(int kernel, int64_t tiles, int64_t steps) {
  const FusedCost& c = kCost[kernel];
  const double turns = (double)ceil_div(tiles, 256), rounds = kernel == kTile256 ? turns : tiles / 512.0;
  const double filling = kernel <= kDecode64 ? 0.25 * rounds + 0.375 * turns : rounds;
  return c.launch + rounds * c.round + (double)steps * std::max(c.first, filling * c.step);
}

static FusedPlan cheapest(int64_t M, int64_t NB, int64_t KP, bool swiglu) {
  const int64_t KB = ceil_div(KP, 2);
  FusedPlan best{kTile64, 1, false};
  double least = 1e300;
  for (int k = kDecode16; k <= kTile256; ++k) {
    const FusedCost& c = kCost[k];
    if (k == kDecode16 && swiglu) continue;           // pairs of blocks
    // never the best, and the low tiles' grids have limits
    if ((k <= kTile32 && M > c.rows * 128) || (k > kTile64 && c.rows >= 4 * M)) continue;
    if (k == kTile256 && KP <= 2) continue;           // its pipeline is two steps deep
    const int64_t tiles = ceil_div(M, c.rows) * ceil_div(NB * 16, c.cols);
    auto consider = [&](int64_t S) {
      const int64_t per = ceil_div(KB, S);
      S = ceil_div(KB, per);  // no empty part
      const int64_t n = tiles * S;
      double t = tiles_time(k, n, per);
      if (S > 1) t += c.join + c.part * (double)(n * c.rows * c.cols * 4) * 1e-6;
      if (t < least) {
        least = t;
        best = FusedPlan{k, (int)S, false};
      }
    };
    consider(1);
    if (k != kTile32 && k != kTile64 && k != kTile128) continue;  // (64 x 256 gained nothing)
    for (const int64_t slots : {128, 256, 512}) {
      const int64_t S = slots / tiles;
      if (S >= 2 && KB >= 3 * S) consider(S);
    }
  }
  return best;
}

// Copied first: rows of less than a load, and rows that wide tiles cannot copy by DMA. (The
// other kernels load any address: BF16 300 x 1000 x 5761 16.9 us, with a copy 17.0; K 5760
// 15.7.)
static int64_t copy_bytes(int64_t M, int64_t kbytes) { return round_up(round_up(kbytes, kStepBytes) * M, 256); }

// sums of the parts of K
static int64_t part_bytes(const FusedPlan& plan, int64_t M, int64_t NB) {
  if (plan.S == 1) return 0;
  const FusedCost& c = kCost[plan.kernel];
  return (int64_t)plan.S * round_up(M, c.rows) * round_up(NB * 16, c.cols) * 4;
}

FusedPlan fused_plan(const FusedGemm& p) {
  FusedPlan plan = cheapest(p.M, p.NB, p.KP, p.act == W8A8_ACT_SWIGLU);
  plan.copy = p.kbytes < 16 || (plan.kernel == kTile256 && !fused_rows_ok(p));
  return plan;
}

void fused_tile(const FusedPlan& plan, int32_t* rows, int32_t* cols) {
  *rows = kCost[plan.kernel].rows;
  *cols = kCost[plan.kernel].cols;
}

int64_t fused_room_bytes(const FusedGemm& p, const FusedPlan& plan) {
  return (plan.copy ? copy_bytes(p.M, p.kbytes) : 0) + part_bytes(plan, p.M, p.NB);
}

// Never falls as M grows, so that a room made for the most rows serves every batch. A plan
// depends on the rows through ceil(M / 16) alone, and K is split only where 256 tiles at
// most leave slots: the row counts up to that are gone through (2048 plans at most, 0.3 ms;
// 30 us for 4096 columns). The copy is counted for every M that could come to the wide
// tiles, whether or not their cost takes it there.
int64_t fused_most_bytes(int type, int64_t M, int64_t N, int64_t K) {
  const int64_t kbytes = type == kFusedInt8 ? K : 2 * K;
  const int64_t NB = type == kFusedInt8 ? ceil_div(N, 16) : round_up(N, 32) / 16;
  const int64_t KP = type == kFusedInt8 ? ceil_div(K, 64) : 2 * ceil_div(K, 64);
  int64_t most = kbytes < 16 || (M > 64 && KP > 2) ? copy_bytes(M, kbytes) : 0;
  int64_t rows = 0;
  for (const int k : {kTile32, kTile64, kTile128})
    rows = std::max(rows, 256 / ceil_div(NB * 16, kCost[k].cols) * kCost[k].rows);
  for (int64_t m = 16; m < std::min(M, rows) + 16; m += 16)
    for (const bool swiglu : {false, true}) {
      const FusedPlan plan = cheapest(m, NB, KP, swiglu);
      most = std::max(most, part_bytes(plan, m, NB));
      if (plan.kernel != kDecode16) break;  // the same for SwiGLU
    }
  return most;
}

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
static void launch_tiles(const FusedGemm& p, int S, void* room, hipStream_t stream) {
  const int64_t mt = ceil_div(p.M, MB * 16), nt = ceil_div(p.NB, 8 * NBW);
  const int per = (int)ceil_div(ceil_div(p.KP, 2), S);
  S = (int)ceil_div(ceil_div(p.KP, 2), per);  // no empty part
  uint8_t* part = reinterpret_cast<uint8_t*>(room);
  hipLaunchKernelGGL((fused_dense_kernel<TY, MB, NBW>), dim3((unsigned)mt, (unsigned)nt, (unsigned)S), dim3(512), 0,
                     stream, p, S, per, part);
  if (S > 1)
    hipLaunchKernelGGL((fused_join_kernel<TY, MB, NBW>), dim3((unsigned)(mt * nt * 2 * MB * NBW)), dim3(256), 0, stream, p,
                       S, (int)mt, mt * nt, part);
}

template <int TY>
static hipError_t launch_dense(const FusedGemm& p, const FusedPlan& plan, void* room, hipStream_t stream) {
  switch (plan.kernel) {
    case kDecode16: launch_decode<TY, 1, 1>(p, stream); break;
    case kDecode16x32: launch_decode<TY, 1, 2>(p, stream); break;
    case kDecode32: launch_decode<TY, 2, 2>(p, stream); break;
    case kDecode64: launch_decode<TY, 4, 2>(p, stream); break;
    case kTile32: launch_tiles<TY, 2, 1>(p, plan.S, room, stream); break;
    case kTile64: launch_tiles<TY, 4, 1>(p, plan.S, room, stream); break;
    case kTile64x256: launch_tiles<TY, 4, 2>(p, plan.S, room, stream); break;
    case kTile128: launch_tiles<TY, 8, 2>(p, plan.S, room, stream); break;
    case kTile256: {
      const int64_t tiles = ceil_div(p.M, 256) * ceil_div(p.NB, 16);
      hipLaunchKernelGGL(fused_wide_kernel<TY>, dim3((unsigned)std::min<int64_t>(256, round_up(tiles, 8))), dim3(512), 0,
                         stream, p);
      break;
    }
  }
  return hipGetLastError();
}

// Rows of a grouped product's tiles (128 rows: of 256 columns, 64: of 128), from the most
// tiles that there can be, by the cost of a dense product of as many. In us, 64 and 128:
// 1003 rows, 7 experts of 1412 x 1000 17.4, 37.8; 128 rows, 256 experts of 4096 x 4096 524,
// 546; 8192 rows, 16 experts of 2048 x 2048 126, 120; 16384 rows, 64 experts of 4096 x 4096
// 1273, 743.
static int grouped_rows(int64_t R, int64_t E, int64_t NB, int64_t KP) {
  double t[2];
  for (int i = 0; i < 2; ++i) {
    const int k = i ? kTile128 : kTile64;
    const FusedCost& c = kCost[k];
    t[i] = tiles_time(k, max_tiles(R, E, c.rows) * ceil_div(NB * 16, c.cols), ceil_div(KP, 2));
  }
  return kCost[t[1] < t[0] ? kTile128 : kTile64].rows;
}

static int64_t grouped_columns(int64_t NB, int tile_rows) { return ceil_div(NB, tile_rows == kTileRows ? 16 : 8); }

static int64_t blocks_of(int64_t N) { return round_up(N, 32) / 16; }
static int64_t pieces_of(int64_t K) { return 2 * ceil_div(K, 64); }

int64_t fused_sched_bytes(int64_t R, int64_t E, int64_t N, int64_t K) {
  return 256 + 16 * max_tiles(R, E, grouped_rows(R, E, blocks_of(N), pieces_of(K)));
}

// the list of the low tiles, the longest: taller ones begin at some row count
int64_t fused_most_sched_bytes(int64_t R, int64_t E) { return 256 + 16 * max_tiles(R, E, kCost[kTile64].rows); }

int64_t fused_grid(int64_t R, int64_t E, int64_t N, int64_t K) {
  const int rows = grouped_rows(R, E, blocks_of(N), pieces_of(K));
  return round_up(max_tiles(R, E, rows), 8) * grouped_columns(blocks_of(N), rows);
}

// Wide tiles for experts of many rows: two steps of K, rows as they copy them, 32-bit
// offsets from a's first row where rows are read through an index.
static bool grouped_wide(const FusedGemm& p, int rows) {
  return rows == kTileRows && p.KP > 2 && fused_rows_ok(p) && (!p.row_index || p.a_rows * p.lda < (int64_t)1 << 32);
}

void fused_grouped_tile(const FusedGemm& p, int32_t* rows, int32_t* cols) {
  const int low = grouped_rows(p.M, p.E, p.NB, p.KP);
  *rows = grouped_wide(p, low) ? kWideRows : low;
  *cols = low == kTileRows ? 256 : 128;
}

hipError_t launch_fused_grouped(const FusedGemm& p, void* ws, hipStream_t stream) {
  const int rows = grouped_rows(p.M, p.E, p.NB, p.KP);
  const bool wide = grouped_wide(p, rows);
  hipLaunchKernelGGL(fused_schedule_kernel, dim3(1), dim3(256), 0, stream, p.group_list, (int)p.E, p.M, (int)wide, rows,
                     reinterpret_cast<int*>(ws), reinterpret_cast<int4*>(reinterpret_cast<char*>(ws) + 256));
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int64_t NT = grouped_columns(p.NB, rows), grid = round_up(max_tiles(p.M, p.E, rows), 8) * NT;
  auto fn = rows == kTileRows ? fused_grouped_kernel<kFusedBf16, 2> : fused_grouped_kernel<kFusedBf16, 1>;
  hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(512), 0, stream, p, (int)NT);
  return hipGetLastError();
}

hipError_t launch_fused_gemm(FusedGemm p, const FusedPlan& plan, void* room, hipStream_t stream) {
  if (plan.copy) {
    const int64_t per = round_up(p.kbytes, kStepBytes) / 16;
    uint8_t* rows = reinterpret_cast<uint8_t*>(room);
    hipLaunchKernelGGL(fused_copy_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(p.M * per, 256), 1 << 16)), dim3(256),
                       0, stream, p.a, p.M, p.lda, p.kbytes, per, rows);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    room = rows + copy_bytes(p.M, p.kbytes);
    p.a = rows;
    p.lda = p.kbytes = per * 16;
  }
  return p.type == kFusedInt8 ? launch_dense<kFusedInt8>(p, plan, room, stream)
                              : launch_dense<kFusedBf16>(p, plan, room, stream);
}

}  // namespace w8a8
