// Attention of packed prompts (moe_attn_prefill of the C ABI): arguments and
// launcher.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8moe {

struct PrefillArgs {
  const __nv_bfloat16 *q, *k, *v;  // head rows: head h of token t at t * stride + h * d
  int64_t q_stride, k_stride, v_stride;
  int Tq, Tk;
  const int32_t *q_starts, *k_starts;  // [B + 1]
  int B, n_heads, n_kv;
  float scale, softcap;
  const float *slopes;
  int window, causal;
  __nv_bfloat16 *out;
  int64_t out_stride;
  float *lse;
  int *err;
  uint64_t wait_ns;  // the limit of a wait
  // The query heads of a key/value head are taken `heads` at a time, in `chunks`
  // pieces; a tile's 128 rows are the heads of `tokens` tokens.
  int heads, chunks, tokens;
  int64_t items;  // tiles at most, times n_kv * chunks; below 2^31
  int stride;     // items between one and the next of a block; 0: asked for
  int splits;     // CTAs of a cluster that share an item's blocks; 1: a block of the launch has whole ones
};
// Clusters of 2, 4, 8 and 16 that are resident together.
constexpr int kSplitSizes = 4;
struct PrefillFit {
  int clusters[kSplitSizes] = {};
};
// Fills in heads, chunks, tokens, items and splits, for so many SMs.
void plan_prefill(PrefillArgs *a, int d, int sms, const PrefillFit &fit);
// Readies the kernels of d whose weights keep 8 or 16 bits.
cudaError_t ready_prefill(int d, int bits, PrefillFit *fit);
// sms: the SMs it may fill, 0 for all.
cudaError_t launch_prefill(const PrefillArgs &a, int d, int bits, int sms, cudaStream_t s);

}  // namespace fp8moe
