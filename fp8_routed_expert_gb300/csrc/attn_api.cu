// C ABI of the attention over a paged key/value cache: context, argument
// checks and launches.  See include/fp8moe.h for the contract.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "common.cuh"
#include "fp8moe.h"
#include "paged_attn.h"

using namespace fp8moe;

// How moe_attn_decode takes the query heads of a key/value head: `group` at a
// time; and by format, the CTAs that are resident, the positions of a tile, the
// warps of a CTA, and the resident clusters of 1, 2, 4 and 8 CTAs.
struct DecodePlan {
  int group = 1;
  int ctas[2] = {0, 0}, tile[2] = {1, 1}, warps[2] = {1, 1}, clusters[2][4] = {};
};

struct moe_attn {
  moe_attn_config cfg{};
  char *ws = nullptr;         // one allocation, the views below
  int sms = 0;                // of the device
  int *err = nullptr;
  uint64_t *turns = nullptr;  // [rope_dim / 2]
  DecodePlan wide, narrow;    // groups as large as may be, and of 8 heads at most
  // moe_attn_decode's workspace
  int group = 1, max_ctas = 0;
  int *counters = nullptr;    // [3][max_ctas], zero between calls
  float *part_ml = nullptr;   // [2 * max_ctas][group][2]
  float *part = nullptr;      // [2 * max_ctas][group][head_dim]
  cudaStream_t last_stream = nullptr;
};

namespace {

#define ATTN_TRY(x)                              \
  do {                                           \
    if ((x) != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxBatch = 1 << 20;
constexpr int64_t kMaxPositions = 0x7fffffff - 63;
constexpr int64_t kMaxTokens = 0x7fffffff;
constexpr int64_t kMaxStride = INT64_C(1) << 40;

int check_config(const moe_attn_config &c) {
  if (c.n_kv_heads < 1 || c.n_heads < c.n_kv_heads || c.n_heads > 1024 ||
      c.n_heads % c.n_kv_heads != 0)
    return MOE_ERR_SHAPE;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return MOE_ERR_SHAPE;
  if (c.rope_dim < 0 || c.rope_dim > c.head_dim || c.rope_dim % 16 != 0) return MOE_ERR_SHAPE;
  if (c.max_sms < 0 || c.device < 0) return MOE_ERR_SHAPE;
  if (c.interleaved != 0 && c.interleaved != 1) return MOE_ERR_ARG;
  if (c.rope_dim > 0 && c.rope_freqs == nullptr) return MOE_ERR_ARG;
  for (int i = 0; i < c.rope_dim / 2; ++i)
    if (!std::isfinite(c.rope_freqs[i])) return MOE_ERR_ARG;
  return MOE_OK;
}

// freq / (2 pi) modulo 1 in units of 2^-64 turns.  1 / (2 pi) is held as the
// sum of two doubles, and the product's rounding error is recovered with an
// fma, so the result is within a unit for |freq| <= 1.  A negative frequency's
// fraction would be rounded to 2^-53: it is the opposite of the positive one's.
uint64_t turns_of(double freq) {
  if (freq < 0.0) return 0 - turns_of(-freq);
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const double p = freq * kHi;
  const double e = std::fma(freq, kHi, -p) + freq * kLo;
  const double f = p - std::floor(p);  // exact, in [0, 1)
  // the fraction's high and low 32 bits, then the (signed) remainder
  const double hi = std::floor(std::ldexp(f, 32));
  const double lo = std::ldexp(std::ldexp(f, 32) - hi, 32);
  const double r = std::ldexp(std::remainder(e, 1.0), 32);  // in [-2^31, 2^31]
  const double rhi = std::floor(r), rlo = std::ldexp(r - rhi, 32);
  return ((uint64_t)hi << 32) + (uint64_t)std::nearbyint(lo) + ((uint64_t)(int64_t)rhi << 32) +
         (uint64_t)std::nearbyint(rlo);
}

// moe_attn_decode's groups of a key/value head, and tiles of all sequences at
// the longest.
int groups_of(const DecodePlan &p, const moe_attn_config &c) {
  return (c.n_heads / c.n_kv_heads + p.group - 1) / p.group;
}
int64_t list_tiles(const DecodePlan &p, int format, const moe_attn_config &c, const DecodeArgs &r) {
  const int tile = p.tile[format];
  return (int64_t)r.B * c.n_kv_heads * groups_of(p, c) * ((r.capacity + tile - 1) / tile);  // < 2^62
}

// Sets *r to clusters of CTAs per segment and returns their grid, or 0 where the
// list of tiles is better or a warp would have more than `limit` tiles.  As many
// CTAs as give each warp a tile of the longest sequence, 32 warps at most, and no
// more than are resident; where a warp would have more than 4 tiles, several
// clusters share a segment, so that it has 3, but no more than 8/9 of the clusters
// that fit, since those that wait for the launch before to leave come too late.
// The list, which balances lengths and uses all SMs, is better where a warp would
// have more than 8 tiles, 16 of a sequence alone, or 4 with clusters on less than
// a third of the SMs.  Four heads of 128 elements per key/value head, bf16, list
// against clusters:
//   one sequence of 2000, 8 key/value heads    11.1 us,  7.0 (2 tiles per warp)
//   of 8000                                    15.5,    11.4
//   of 16000                                   21.6,    17.2
//   of 64000                                   47.1,    44.4 (16)
//   of 4000, 4 key/value heads (32 CTAs)       11.8,     9.0 (4)
//   4 sequences of up to 16000, 4 heads        23.2,    20.3 (8)
//   of up to 32000                             32.4,    33.4 (16)
//   32 sequences of up to 500, 8 heads         11.9,     9.8 (4, clusters of one)
int take_clusters(const moe_attn *a, const DecodePlan &p, int format, int64_t limit, DecodeArgs *r) {
  r->group = p.group;
  r->groups_per_kv = groups_of(p, a->cfg);
  r->n_groups = a->cfg.n_kv_heads * r->groups_per_kv;
  const int tile = p.tile[format], warps = p.warps[format];
  const int *fit = p.clusters[format];
  const int64_t per_segment = (r->capacity + tile - 1) / tile, segments = (int64_t)r->B * r->n_groups;
  int k = 0;
  while (k < 3 && (warps << k) < 32 && (warps << k) < per_segment && segments <= fit[k + 1]) ++k;
  if (segments > fit[k]) return 0;
  const int64_t wide = warps << k;
  int64_t splits = 1;
  if (per_segment > 4 * wide)
    splits = std::max<int64_t>(
        1, std::min((per_segment + 3 * wide - 1) / (3 * wide), (fit[k] - fit[k] / 9) / segments));
  const int64_t most = 3 * (splits * segments << k) < a->sms ? 4 : r->B == 1 ? 16 : 8;
  if (per_segment > std::min(most, limit) * wide * splits) return 0;
  r->cluster = 1 << k;
  r->splits = (int)splits;
  return (int)(splits * segments << k);
}

// Chooses how moe_attn_decode splits a call with r->B and r->capacity, and returns
// the grid; r->cluster is 0 for the list of tiles.
// More than 8 heads per key/value head: where clusters have few tiles per warp,
// groups of 8, which read the rows again from L2, are faster than the products of
// up to 16 heads in a warp.  16 heads of 128 elements, bf16, list against clusters
// of groups of 8 and of 16:
//   one sequence of 1000, 1 key/value head      -,      5.7,  8.9 us
//   of 16000                                   15.1,   10.3, 14.6
//   of 64000                                   20.0,   17.3, 18.1
//   of 128000                                  26.1,   23.4, 22.3 (7 and 4 tiles per warp)
//   of 32000, 4 key/value heads                27.5,   22.2, 19.7 (7 and 8)
//   2 of up to 64000, 2 heads of 64 elements   17.7,     -,  19.1
int split_decode(const moe_attn *a, int format, DecodeArgs *r) {
  int grid = 0;
  if (a->narrow.group < a->wide.group) grid = take_clusters(a, a->narrow, format, 4, r);
  if (grid == 0) grid = take_clusters(a, a->wide, format, 16, r);
  if (grid == 0) grid = (int)std::min<int64_t>(list_tiles(a->wide, format, a->cfg, *r), a->wide.ctas[format]);
  return grid;
}

// The caller's cache, checked against the context, as the kernels take it.
int view_of(const moe_attn *a, const moe_paged_kv *kv, KvView *v) {
  if (kv == nullptr) return MOE_ERR_ARG;
  if (kv->format != MOE_KV_BF16 && kv->format != MOE_KV_E4M3) return MOE_ERR_ARG;
  const bool q = kv->format == MOE_KV_E4M3;
  if (kv->n_pages < 1 || kv->n_pages > 0x7fffffff || kv->page_size < 1) return MOE_ERR_SHAPE;
  if (kv->k == nullptr || kv->v == nullptr) return MOE_ERR_ARG;
  if (q && (kv->k_scale == nullptr || kv->v_scale == nullptr)) return MOE_ERR_ARG;
  const int es = q ? 1 : 2;
  // Every offset in bytes is kept within 62 bits: strides alone do not, 2^31 pages
  // of 2^41 bytes would wrap to another address.
  const auto far = [&](int64_t page, int64_t head, int64_t slot, int64_t row, int bytes) {
    return ((__int128)(kv->n_pages - 1) * page + (__int128)(a->cfg.n_kv_heads - 1) * head +
            (__int128)(kv->page_size - 1) * slot + row) * bytes > INT64_C(1) << 62;
  };
  for (int64_t st : {kv->page_stride, kv->head_stride, kv->slot_stride}) {
    if (st < 0 || st > kMaxStride) return MOE_ERR_SHAPE;
    if ((st * es) % 16 != 0) return MOE_ERR_ALIGN;
  }
  if (far(kv->page_stride, kv->head_stride, kv->slot_stride, a->cfg.head_dim, es)) return MOE_ERR_SHAPE;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return MOE_ERR_ALIGN;
  if (q) {
    for (int64_t st : {kv->scale_page_stride, kv->scale_head_stride, kv->scale_slot_stride})
      if (st < 0 || st > kMaxStride) return MOE_ERR_SHAPE;
    if (far(kv->scale_page_stride, kv->scale_head_stride, kv->scale_slot_stride, 1, 4)) return MOE_ERR_SHAPE;
    if (!aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4)) return MOE_ERR_ALIGN;
  }
  *v = KvView{static_cast<uint8_t *>(kv->k),
              static_cast<uint8_t *>(kv->v),
              q ? kv->k_scale : nullptr,
              q ? kv->v_scale : nullptr,
              kv->n_pages,
              kv->page_stride * es,
              kv->head_stride * es,
              kv->slot_stride * es,
              q ? kv->scale_page_stride : 0,
              q ? kv->scale_head_stride : 0,
              q ? kv->scale_slot_stride : 0,
              kv->page_size};
  return MOE_OK;
}

// Head rows of T tokens: `heads` rows of d elements within each stride.
int check_rows(const void *p, int64_t stride, int heads, int d) {
  if (p == nullptr) return MOE_ERR_ARG;
  if (stride < (int64_t)heads * d || stride > (INT64_C(1) << 31)) return MOE_ERR_SHAPE;
  if (!aligned(p, 16) || stride % 8 != 0) return MOE_ERR_ALIGN;
  return MOE_OK;
}

int check_norm(const moe_attn *a, const int32_t *positions, const float *wq, const float *wk,
               float eps) {
  if (a->cfg.rope_dim > 0 && positions == nullptr) return MOE_ERR_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return MOE_ERR_ARG;
  if (!aligned(positions, 4) || !aligned(wq, 16) || !aligned(wk, 16)) return MOE_ERR_ALIGN;
  return MOE_OK;
}

int check_T(const moe_attn *a, int64_t T) {
  if (a == nullptr || T < 0) return MOE_ERR_ARG;
  return T > kMaxTokens ? MOE_ERR_SHAPE : MOE_OK;
}

#define CHECK(x)                  \
  do {                            \
    const int rc_ = (x);          \
    if (rc_ != MOE_OK) return rc_; \
  } while (0)

int run_rows(moe_attn *a, RowArgs &r, cudaStream_t s) {
  r.sms = a->sms;
  r.err = a->err;
  ATTN_TRY(cudaSetDevice(a->cfg.device));
  a->last_stream = s;
  ATTN_TRY(launch_rows(r, a->cfg.head_dim, s));
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_attn_init(moe_attn **out, const moe_attn_config *cfg) {
  if (out == nullptr) return MOE_ERR_ARG;
  *out = nullptr;
  if (cfg == nullptr) return MOE_ERR_ARG;
  CHECK(check_config(*cfg));
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || cfg->device >= count) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  if (cudaSetDevice(cfg->device) != cudaSuccess) return MOE_ERR_CUDA;
  int major = 0, minor = 0, sms = 0;
  ATTN_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, cfg->device));
  ATTN_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, cfg->device));
  ATTN_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, cfg->device));
  if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED;
  moe_attn *a = new (std::nothrow) moe_attn();
  if (a == nullptr) return MOE_ERR_NOMEM;
  a->cfg = *cfg;
  a->cfg.rope_freqs = nullptr;  // the caller's array is not kept
  a->sms = sms;
  const int use = cfg->max_sms > 0 && cfg->max_sms < sms ? cfg->max_sms : sms;
  const int per_kv = cfg->n_heads / cfg->n_kv_heads;
  a->wide.group = decode_group(per_kv, cfg->head_dim, false);
  a->narrow.group = decode_group(per_kv, cfg->head_dim, true);
  a->group = a->wide.group;
  for (DecodePlan *plan : {&a->wide, &a->narrow})
    for (int f = 0; f < 2; ++f) {
      int per_sm = 0;
      if (plan_paged_decode(cfg->head_dim, f == MOE_KV_E4M3, plan->group, &per_sm, &plan->tile[f],
                            &plan->warps[f], plan->clusters[f]) != cudaSuccess ||
          per_sm < 1) {
        cudaGetLastError();
        delete a;
        return MOE_ERR_CUDA;
      }
      plan->ctas[f] = per_sm * use;
      plan->clusters[f][0] = plan->ctas[f];
      for (int i = 1; i < 4; ++i)
        plan->clusters[f][i] = std::min(plan->clusters[f][i], plan->ctas[f] >> i);
      a->max_ctas = std::max(a->max_ctas, plan->ctas[f]);
    }
  const int half = cfg->rope_dim / 2;
  uint64_t turns[128];
  for (int i = 0; i < half; ++i) turns[i] = turns_of(cfg->rope_freqs[i]);
  auto up256 = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t n = (size_t)a->max_ctas, g = (size_t)a->group;
  const size_t b_counters = up256(3 * n * sizeof(int)), b_ml = up256(2 * n * g * 2 * sizeof(float));
  const size_t b_part = up256(2 * n * g * (size_t)cfg->head_dim * sizeof(float));
  const size_t cleared = 256 + up256(sizeof(turns)) + b_counters;
  if (cudaMalloc(&a->ws, cleared + b_ml + b_part) != cudaSuccess) {
    cudaGetLastError();
    delete a;
    return MOE_ERR_NOMEM;
  }
  char *p = a->ws;
  a->err = reinterpret_cast<int *>(p);
  a->turns = reinterpret_cast<uint64_t *>(p += 256);
  a->counters = reinterpret_cast<int *>(p += up256(sizeof(turns)));
  a->part_ml = reinterpret_cast<float *>(p += b_counters);
  a->part = reinterpret_cast<float *>(p += b_ml);
  if (cudaMemset(a->ws, 0, cleared) != cudaSuccess ||
      cudaMemcpy(a->turns, turns, (size_t)half * sizeof(uint64_t), cudaMemcpyHostToDevice) !=
          cudaSuccess ||
      cudaDeviceSynchronize() != cudaSuccess) {  // ready for any stream
    moe_attn_free(a);
    return MOE_ERR_CUDA;
  }
  *out = a;
  return MOE_OK;
}

void moe_attn_free(moe_attn *a) {
  if (a == nullptr) return;
  cudaSetDevice(a->cfg.device);
  if (a->ws) cudaFree(a->ws);
  delete a;
}

int moe_attn_status(moe_attn *a) {
  if (a == nullptr) return MOE_ERR_ARG;
  ATTN_TRY(cudaSetDevice(a->cfg.device));
  ATTN_TRY(cudaStreamSynchronize(a->last_stream));
  int flag = 0;
  ATTN_TRY(cudaMemcpy(&flag, a->err, sizeof(int), cudaMemcpyDeviceToHost));
  ATTN_TRY(cudaMemset(a->err, 0, sizeof(int)));
  // a kernel on a stream that does not wait for the default one must find it cleared
  ATTN_TRY(cudaStreamSynchronize(nullptr));
  return flag ? MOE_ERR_DEVICE : MOE_OK;
}

int moe_attn_norm_rope(moe_attn *a, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                       const int32_t *positions, int64_t T, const float *q_weight,
                       const float *k_weight, float eps, void *q_out, int64_t q_out_stride,
                       void *k_out, int64_t k_out_stride, void *stream) {
  CHECK(check_T(a, T));
  if (T == 0) return MOE_OK;
  const moe_attn_config &c = a->cfg;
  CHECK(check_rows(q, q_stride, c.n_heads, c.head_dim));
  CHECK(check_rows(k, k_stride, c.n_kv_heads, c.head_dim));
  CHECK(check_rows(q_out, q_out_stride, c.n_heads, c.head_dim));
  CHECK(check_rows(k_out, k_out_stride, c.n_kv_heads, c.head_dim));
  CHECK(check_norm(a, positions, q_weight, k_weight, eps));
  RowArgs r{};
  r.q = {static_cast<const __nv_bfloat16 *>(q), q_stride};
  r.k = {static_cast<const __nv_bfloat16 *>(k), k_stride};
  r.q_out = {static_cast<__nv_bfloat16 *>(q_out), q_out_stride};
  r.k_out = {static_cast<__nv_bfloat16 *>(k_out), k_out_stride};
  r.n_q = c.n_heads;
  r.n_k = c.n_kv_heads;
  r.T = T;
  r.positions = positions;
  r.q_weight = q_weight;
  r.k_weight = k_weight;
  r.turns = a->turns;
  r.half = c.rope_dim / 2;
  r.interleaved = c.interleaved;
  r.eps = eps;
  return run_rows(a, r, static_cast<cudaStream_t>(stream));
}

int moe_attn_append(moe_attn *a, const moe_paged_kv *kv, const void *q, int64_t q_stride,
                    const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                    const int32_t *positions, const int64_t *slots, int64_t T,
                    const float *q_weight, const float *k_weight, float eps, void *q_out,
                    int64_t q_out_stride, void *stream) {
  CHECK(check_T(a, T));
  RowArgs r{};
  CHECK(view_of(a, kv, &r.kv));
  if (T == 0) return MOE_OK;
  const moe_attn_config &c = a->cfg;
  CHECK(check_rows(q, q_stride, c.n_heads, c.head_dim));
  CHECK(check_rows(k, k_stride, c.n_kv_heads, c.head_dim));
  CHECK(check_rows(v, v_stride, c.n_kv_heads, c.head_dim));
  CHECK(check_rows(q_out, q_out_stride, c.n_heads, c.head_dim));
  CHECK(check_norm(a, positions, q_weight, k_weight, eps));
  if (slots == nullptr) return MOE_ERR_ARG;
  if (!aligned(slots, 8)) return MOE_ERR_ALIGN;
  r.q = {static_cast<const __nv_bfloat16 *>(q), q_stride};
  r.k = {static_cast<const __nv_bfloat16 *>(k), k_stride};
  r.v = {static_cast<const __nv_bfloat16 *>(v), v_stride};
  r.q_out = {static_cast<__nv_bfloat16 *>(q_out), q_out_stride};
  r.n_q = c.n_heads;
  r.n_k = r.n_v = c.n_kv_heads;
  r.T = T;
  r.positions = positions;
  r.slots = slots;
  r.q_weight = q_weight;
  r.k_weight = k_weight;
  r.turns = a->turns;
  r.half = c.rope_dim / 2;
  r.interleaved = c.interleaved;
  r.eps = eps;
  r.cache = true;
  r.e4m3 = kv->format == MOE_KV_E4M3;
  return run_rows(a, r, static_cast<cudaStream_t>(stream));
}

int moe_attn_write(moe_attn *a, const moe_paged_kv *kv, const void *k, int64_t k_stride,
                   const void *v, int64_t v_stride, const int64_t *slots, int64_t T, void *stream) {
  CHECK(check_T(a, T));
  RowArgs r{};
  CHECK(view_of(a, kv, &r.kv));
  if (T == 0) return MOE_OK;
  const moe_attn_config &c = a->cfg;
  CHECK(check_rows(k, k_stride, c.n_kv_heads, c.head_dim));
  CHECK(check_rows(v, v_stride, c.n_kv_heads, c.head_dim));
  if (slots == nullptr) return MOE_ERR_ARG;
  if (!aligned(slots, 8)) return MOE_ERR_ALIGN;
  r.k = {static_cast<const __nv_bfloat16 *>(k), k_stride};
  r.v = {static_cast<const __nv_bfloat16 *>(v), v_stride};
  r.n_k = r.n_v = c.n_kv_heads;
  r.T = T;
  r.slots = slots;
  r.cache = true;
  r.e4m3 = kv->format == MOE_KV_E4M3;
  return run_rows(a, r, static_cast<cudaStream_t>(stream));
}

int moe_attn_read(moe_attn *a, const moe_paged_kv *kv, const int64_t *slots, int64_t T, void *k_out,
                  int64_t k_out_stride, void *v_out, int64_t v_out_stride, void *stream) {
  CHECK(check_T(a, T));
  ReadArgs r{};
  CHECK(view_of(a, kv, &r.kv));
  if (T == 0) return MOE_OK;
  const moe_attn_config &c = a->cfg;
  CHECK(check_rows(k_out, k_out_stride, c.n_kv_heads, c.head_dim));
  CHECK(check_rows(v_out, v_out_stride, c.n_kv_heads, c.head_dim));
  if (slots == nullptr) return MOE_ERR_ARG;
  if (!aligned(slots, 8)) return MOE_ERR_ALIGN;
  r.e4m3 = kv->format == MOE_KV_E4M3;
  r.slots = slots;
  r.T = T;
  r.n_kv = c.n_kv_heads;
  r.k_out = {static_cast<__nv_bfloat16 *>(k_out), k_out_stride};
  r.v_out = {static_cast<__nv_bfloat16 *>(v_out), v_out_stride};
  r.sms = a->sms;
  r.err = a->err;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  ATTN_TRY(cudaSetDevice(c.device));
  a->last_stream = s;
  ATTN_TRY(launch_read(r, c.head_dim, s));
  return MOE_OK;
}

int moe_attn_decode_clusters(const moe_attn *a, const moe_paged_kv *kv, int64_t B, int64_t max_pages) {
  if (a == nullptr || B < 0) return MOE_ERR_ARG;
  if (B > kMaxBatch) return MOE_ERR_SHAPE;
  DecodeArgs r{};
  CHECK(view_of(a, kv, &r.kv));
  if (max_pages < (B > 0 ? 1 : 0) || max_pages > kMaxPositions / kv->page_size) return MOE_ERR_SHAPE;
  if (B == 0) return 0;
  r.B = (int)B;
  r.capacity = max_pages * kv->page_size;
  if (list_tiles(a->wide, kv->format, a->cfg, r) > INT64_C(1) << 29) return MOE_ERR_SHAPE;
  split_decode(a, kv->format, &r);
  return r.cluster > 0 ? r.splits : 0;
}

int moe_attn_decode(moe_attn *a, const moe_paged_kv *kv, const void *q, int64_t q_stride,
                    const int32_t *page_table, int64_t table_stride, int64_t max_pages,
                    const int32_t *seq_lens, const int32_t *starts, int64_t B, float scale,
                    float softcap, const float *slopes, int32_t window, void *out, float *lse,
                    void *stream) {
  if (a == nullptr || B < 0) return MOE_ERR_ARG;
  if (B > kMaxBatch) return MOE_ERR_SHAPE;
  DecodeArgs r{};
  CHECK(view_of(a, kv, &r.kv));
  if (max_pages < (B > 0 ? 1 : 0) || max_pages > kMaxPositions / kv->page_size || table_stride < 0 ||
      table_stride > kMaxStride)
    return MOE_ERR_SHAPE;
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0)
    return MOE_ERR_ARG;
  if (B == 0) return MOE_OK;
  const moe_attn_config &c = a->cfg;
  CHECK(check_rows(q, q_stride, c.n_heads, c.head_dim));
  if (!page_table || !seq_lens || !out) return MOE_ERR_ARG;
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(starts, 4) ||
      !aligned(slopes, 4) || !aligned(out, 16) || !aligned(lse, 4))
    return MOE_ERR_ALIGN;
  r.q = static_cast<const __nv_bfloat16 *>(q);
  r.q_stride = q_stride;
  r.table = page_table;
  r.table_stride = table_stride;
  r.capacity = max_pages * kv->page_size;
  r.lens = seq_lens;
  r.starts = starts;
  r.B = (int)B;
  r.n_heads = c.n_heads;
  r.n_kv = c.n_kv_heads;
  r.part = a->part;
  r.part_ml = a->part_ml;
  r.counters = a->counters;
  r.max_ctas = a->max_ctas;
  r.scale = scale;
  r.softcap = softcap;
  r.slopes = slopes;
  r.window = window;
  r.out = static_cast<__nv_bfloat16 *>(out);
  r.lse = lse;
  r.err = a->err;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  ATTN_TRY(cudaSetDevice(c.device));
  a->last_stream = s;
  decode_page_division(&r);
  if (list_tiles(a->wide, kv->format, c, r) > INT64_C(1) << 29) return MOE_ERR_SHAPE;
  const int grid = split_decode(a, kv->format, &r);
  ATTN_TRY(launch_paged_decode(r, c.head_dim, kv->format == MOE_KV_E4M3, grid, s));
  return MOE_OK;
}

}  // extern "C"
