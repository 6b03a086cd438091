// Kernels of the attention over a paged key/value cache (moe_attn_* of the C
// ABI): arguments and launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fp8moe {

// The caller's cache: strides in bytes for the rows, in elements for the
// scales (moe_paged_kv).
struct KvView {
  uint8_t *k, *v;
  float *k_scale, *v_scale;  // null for bf16
  int64_t n_pages;
  int64_t page_stride, head_stride, slot_stride;
  int64_t scale_page_stride, scale_head_stride, scale_slot_stride;
  int page_size;
};

// bf16 head rows of T tokens: head h of token t at t * stride + h * d.
struct RowsIn {
  const __nv_bfloat16 *p;
  int64_t stride;
};
struct RowsOut {
  __nv_bfloat16 *p;
  int64_t stride;
};

// Norm, rotation and storing of head rows.  A token has n_q query rows, n_k
// key rows and n_v value rows; with a cache, key and value rows go there,
// otherwise key rows go to k_out.
struct RowArgs {
  RowsIn q, k, v;
  RowsOut q_out, k_out;
  int n_q, n_k, n_v;
  int64_t T;
  const int32_t *positions;
  const int64_t *slots;
  const float *q_weight, *k_weight;  // null: no norm
  const uint64_t *turns;             // [half]: 2^64 * (radians per position / 2 pi), mod 2^64
  int half, interleaved;             // half = R / 2, 0 for no rotation
  float eps;
  KvView kv;
  bool cache, e4m3;
  int sms;  // of the device
  int *err;
};
cudaError_t launch_rows(const RowArgs &a, int d, cudaStream_t s);

struct ReadArgs {
  KvView kv;
  bool e4m3;
  const int64_t *slots;
  int64_t T;
  int n_kv;
  RowsOut k_out, v_out;
  int sms;
  int *err;
};
cudaError_t launch_read(const ReadArgs &a, int d, cudaStream_t s);

struct DecodeArgs {
  KvView kv;
  const __nv_bfloat16 *q;
  int64_t q_stride;
  const int32_t *table;
  int64_t table_stride;
  int64_t capacity;  // positions a row of the page table covers
  const int32_t *lens, *starts;
  int B, n_heads, n_kv;
  // query heads of a key/value head are taken `group` at a time, in
  // groups_per_kv groups; n_groups = n_kv * groups_per_kv
  int group, groups_per_kv, n_groups;
  float scale, softcap;
  const float *slopes;
  int window;
  __nv_bfloat16 *out;
  float *lse;
  // position / page_size = position * page_mul >> page_shift; whole_pages: the
  // page size is a multiple of 16
  uint32_t page_mul;
  int page_shift;
  bool whole_pages;
  int cluster;  // CTAs of a cluster; 0: the list of all tiles is cut over the CTAs
  int splits;   // clusters of a segment
  // workspace: 2 * max_ctas pieces of group * d outputs and group (m, l)
  // pairs, 3 * max_ctas counters (zero between calls)
  float *part, *part_ml;
  int *counters;
  int max_ctas;
  int *err;
};
// Query heads taken at a time when `heads_per_kv` share a key/value head: as many
// as a kernel takes, or (narrow) 8 at most.
int decode_group(int heads_per_kv, int d, bool narrow);
// Fills in page_mul, page_shift and whole_pages.
void decode_page_division(DecodeArgs *a);
// Readies the kernel; tells how many CTAs of it fit on an SM, the positions of
// a tile, the warps of a CTA and how many clusters of 1, 2, 4 and 8 CTAs fit on
// the device.  Launches take at most max_ctas CTAs and at most 2^29 tiles.
cudaError_t plan_paged_decode(int d, bool e4m3, int group, int *ctas_per_sm, int *tile,
                              int *warps, int (&clusters)[4]);
cudaError_t launch_paged_decode(const DecodeArgs &a, int d, bool e4m3, int grid, cudaStream_t s);

}  // namespace fp8moe
