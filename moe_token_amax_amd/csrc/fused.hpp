// Internal launchers of the products with a fused epilogue (host side): INT8 codes,
// and BF16 rows dense and grouped by expert. Arguments are checked by the C ABI layer
// before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8a8 {

enum FusedType { kFusedInt8 = 0, kFusedBf16 = 1 };

// One product y = act(a w^T + bias) + residual.
struct FusedGemm {
  int type;                  // FusedType
  const uint8_t* a;          // rows of kbytes bytes, row stride lda bytes
  int64_t lda, kbytes;
  int64_t a_rows;            // rows of a (dense: M)
  const int32_t* row_index;  // grouped: row of a for every output row, or null (the row itself)
  int64_t M;                 // output rows
  const uint8_t* w;          // 1 KB blocks [e][n / 16][64 bytes of k]
  int64_t NB;                // 16-column blocks of an expert
  int64_t KP;                // 64-byte pieces of K
  int64_t N;                 // weight rows
  const float* a_scale;      // INT8: [M]
  const float* w_scale;      // INT8: [N]
  const uint16_t* bias;      // [N] or null
  int act;                   // w8a8_act; SwiGLU: blocks 2 i are gate rows, 2 i + 1 up rows, N / 2 outputs
  const uint16_t* residual;  // BF16 [M, outputs], row stride ldr, or null
  int64_t ldr;
  void* y;                   // BF16 or (f32) float [M, outputs], row stride ldy
  int64_t ldy;
  int f32;
  const int64_t* group_list; // [E] or null
  int64_t E;
  const void* ws;            // grouped: the tile list
};

int64_t bf16_packed_bytes(int64_t N, int64_t K);  // of one [N, K] weight
// pairs: the halves [0, N / 2) and [N / 2, N) of the rows in alternating 16-row blocks
hipError_t launch_bf16_prepack(const uint16_t* w, int64_t E, int64_t N, int64_t K, bool pairs, void* packed,
                               hipStream_t stream);

// How a dense product runs, chosen from its sizes and alignment.
struct FusedPlan {
  int kernel;  // of fused.hip's
  int S;       // parts of K (tiles)
  bool copy;   // rows copied to whole, aligned, zero-padded steps first
};
FusedPlan fused_plan(const FusedGemm& p);
// rows and columns of its tiles
void fused_tile(const FusedPlan& plan, int32_t* rows, int32_t* cols);
// Workspace: the copied rows, then the sums of the parts; and the most that a product of
// these columns and at most M rows can need, whatever its rows' alignment.
int64_t fused_room_bytes(const FusedGemm& p, const FusedPlan& plan);
int64_t fused_most_bytes(int type, int64_t M, int64_t N, int64_t K);
// M, N >= 1
hipError_t launch_fused_gemm(FusedGemm p, const FusedPlan& plan, void* room, hipStream_t stream);

// Grouped (R = p.M rows): bytes of the tile list, the most that at most R rows can need,
// workgroups, and the launch, which writes the list into p.ws first.
int64_t fused_sched_bytes(int64_t R, int64_t E, int64_t N, int64_t K);
int64_t fused_most_sched_bytes(int64_t R, int64_t E);
int64_t fused_grid(int64_t R, int64_t E, int64_t N, int64_t K);
// rows and columns of the highest tiles that an expert can get
void fused_grouped_tile(const FusedGemm& p, int32_t* rows, int32_t* cols);
hipError_t launch_fused_grouped(const FusedGemm& p, void* ws, hipStream_t stream);

}  // namespace w8a8
