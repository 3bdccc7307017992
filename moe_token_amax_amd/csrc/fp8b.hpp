// Internal launchers of the block-scaled FP8 kernels and of the expert router
// (host side). Arguments are checked by the C ABI layer before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8a8 {

constexpr int64_t kFp8Block = 128;  // values of K (and rows of the weight) under one scale

// act 0: the rows of x [M, K]; act 1: SwiGLU of x = [gate | up] [M, 2K].
// q [M, ldq] with ldq = K rounded up to whole blocks, scale [ceil(K/128)][M]
hipError_t launch_fp8b_quant(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int act, int scale_alg,
                             uint8_t* q, float* scale, hipStream_t stream);

int64_t fp8b_packed_bytes(int64_t N, int64_t K);  // of one [N, K] weight
hipError_t launch_fp8b_prepack(const uint8_t* w, int64_t E, int64_t N, int64_t K, void* packed,
                               hipStream_t stream);

// One product, dense (group_list null) or grouped.
struct Fp8bGemm {
  const uint8_t* a;          // E4M3 rows, row stride lda (a multiple of 16, whole blocks readable)
  int64_t lda;
  const float* a_scale;      // [KB][a_rows]
  int64_t a_rows;            // rows of a (dense: M)
  const int32_t* row_index;  // grouped: row of a for every output row, or null (the row itself)
  int64_t M;                 // output rows
  int64_t KB;                // 128-deep blocks of K
  const uint8_t* w;          // packed weight(s)
  const float* w_scale;      // [E][ceil(N/128)][KB]
  int64_t N;
  const uint16_t* bias;      // [N] or null
  uint16_t* y;               // BF16 [M, N], row stride ldy
  int64_t ldy;
  const int64_t* group_list; // [E] or null
  int64_t E;
  int exact;                 // grouped: products of the codes as BF16, none of them cut
  const void* ws;            // grouped: the schedule written by launch_fp8b_schedule
  // BF16 input quantized inside (launch_fp8b_linear_fused): a = x, lda in elements
  int64_t K;
  int scale_alg;
};
// tiles of the rows of every expert; any number of products over one
// group_list and R share a schedule
int64_t fp8b_sched_bytes(int64_t R, int64_t E);
int64_t fp8b_grid_tiles(int64_t R, int64_t E, int64_t N);  // workgroups of a grouped product's launch
hipError_t launch_fp8b_schedule(const int64_t* group_list, int64_t E, int64_t R, void* ws, hipStream_t stream);
// launch_fp8b_quant (act 0) of M >= 1 rows and launch_fp8b_schedule in one launch
hipError_t launch_fp8b_quant_schedule(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int scale_alg, uint8_t* q,
                                      float* scale, const int64_t* group_list, int64_t E, int64_t R, void* ws,
                                      hipStream_t stream);
hipError_t launch_fp8b_gemm(const Fp8bGemm& p, hipStream_t stream);
bool fp8b_fused_ok(int64_t M, int64_t K);
hipError_t launch_fp8b_linear_fused(const Fp8bGemm& p, hipStream_t stream);

struct GateArgs {
  const void* logits;  // [T, E], row stride ld
  int dtype;           // 0 fp32, 1 BF16, 2 FP16
  int64_t T, ld;
  int E;
  const float* bias;   // [E] or null
  int scoring;         // 0 softmax, 1 sigmoid
  int n_group, topk_group, top_k;
  int renormalize;
  float scale;
  int32_t* ids;        // [T, top_k]
  float* weights;      // [T, top_k]
  // set by the launcher: floats first; 4 logits per load; 4 biases per load
  bool fast, vec, bias_vec;
};
hipError_t launch_gate(const GateArgs& p, hipStream_t stream);

}  // namespace w8a8
