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
cudaError_t launch_norm(const NormArgs &a, int sms, cudaStream_t s);

struct MatmulArgs {
  int64_t M, N, K;
  const float *a_scale;  // of row m and block b: m * a_row + b * a_block
  int64_t a_row, a_block;
  const float *w_scale;  // [ceil(N / 128)][ceil(K / 128)]
  __nv_bfloat16 *out;
  int64_t out_stride;
  bool whole_lines;  // rows of out begin 32-byte aligned
  int blocks;   // ceil(K / 128)
  int64_t tiles;
  int splits;  // CTAs of a cluster, which share a tile's K blocks
  int stages;  // blocks of operands in flight
  int a_rows;  // rows of an activation box
  int *err;
};
// Columns of a tile, CTAs that share it, and their stages.
void split_matmul(int64_t M, int64_t N, int64_t K, int sms, int *columns, int *splits);
int matmul_stages(int64_t M, int columns, int splits);
cudaError_t launch_matmul(const CUtensorMap &a, const CUtensorMap &w, const MatmulArgs &m, int columns, int sms,
                          cudaStream_t s);
cudaError_t ready_matmul();

}  // namespace fp8moe
