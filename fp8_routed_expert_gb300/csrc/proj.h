// Kernels of the projections around the attention and the MoE (moe_proj_* of
// the C ABI): arguments and launchers.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8moe {

constexpr int64_t kNormColumns = 16384;  // the longest row

struct NormArgs {
  const __nv_bfloat16 *x;
  int64_t x_stride;
  const __nv_bfloat16 *residual;  // null: none
  int64_t residual_stride;
  int64_t T;
  int H;
  const float *weight;  // null: no norm
  float eps;
  __nv_bfloat16 *residual_out;  // null without a residual
  int64_t residual_out_stride;
  __nv_bfloat16 *out;  // null: none
  int64_t out_stride;
  uint8_t *codes;  // null: none
  int64_t codes_stride;
  float *scales;  // of row t and block b: t * scale_row + b * scale_block
  int64_t scale_row, scale_block;
};
// limit: the SMs it may fill, 0 for all `sms`.
cudaError_t launch_norm(const NormArgs &a, int sms, int limit, cudaStream_t s);

struct MatmulArgs {
  int64_t M, N, K;
  const float *a_scale;  // of row m and block b: m * a_row + b * a_block
  int64_t a_row, a_block;
  const float *w_scale;  // [ceil(N / 128)][ceil(K / 128)]
  __nv_bfloat16 *out;
  int64_t out_stride;
  bool whole_lines;  // rows of out begin 32-byte aligned
  int blocks;  // ceil(K / 128)
  int *err;
  // plan_matmul's:
  bool few;                       // at most 64 rows: two CTAs per SM
  int columns, splits;            // of a tile; CTAs of a cluster, which share its K blocks
  int64_t tiles, grid;
  int a_rows, a_bytes;            // of an activation box, and what it has of a stage
  int held;                       // rows that a CTA of a cluster adds up
  int stages, sums_at, scales_at, smem;  // blocks in flight; bytes into shared memory, and all of it
};
constexpr int kMostSplits = 8;
// Resident clusters of 1, 2, ... CTAs: for few rows, and for tiles of 64, 128 and 256
// columns.
struct MatmulFit {
  int few[kMostSplits + 1], many[3][kMostSplits + 1];
};
cudaError_t ready_matmul(MatmulFit *fit);
// Fills in the plan for M, N, K (blocks) on `sms` SMs, or on at most `limit` unless that is 0.
void plan_matmul(const MatmulFit &fit, int sms, int limit, MatmulArgs *m);
cudaError_t launch_matmul(const CUtensorMap &a, const CUtensorMap &w, const CUtensorMap &o, const MatmulArgs &m, cudaStream_t s);

}  // namespace fp8moe
