// Attention of packed prompts on the 5th-generation tensor cores (moe_attn_prefill
// of the C ABI).
//
// Rows and tiles.  The query heads that share a key/value head are rows of one
// tile: TMA brings a box of (tokens x heads x 64 elements), which lies in shared
// memory as rows of 128 bytes, token by token.  A tile of 128 rows is 128 / heads
// tokens, so grouped heads read each key and value once for all of them, and the
// diagonal of the causal mask is 128 / heads keys wide instead of 128.
//
// An item is one or two such tiles (two of heads of 64 and 128 elements; one of 256,
// whose output takes half of tensor memory).  Per block of 128 keys (64 with 256
// elements):
//   S = Q K^T     tcgen05.mma kind::f16, both operands in shared memory, f32 in TMEM
//   P = exp2(S * scale - ref)    in registers: one thread per row, no shuffles;
//                 back to TMEM as bf16 over S
//   O += P V      tcgen05.mma with P from TMEM; V as it lies (rows along K)
// The two tiles (or, with one tile, two S buffers of neighbouring blocks) alternate:
// one is in its softmax while the other's products run.
//
// The softmax reference moves only when a score exceeds it by 2^8 (sums then hold
// weights up to 2^8, as exact in f32 as below 1); only then is O read, scaled and
// written back, by the row's own thread.  Weights are rounded to bf16 for the second
// product, the matrix unit's type for bf16 values: 2^-8 of each weight at most, and
// independent from key to key; the sum is of the f32 weights.
//
// Blocks that no row sees are not visited; masks are applied in blocks that not all
// rows see in full.  A hidden value's weight is zero, but zero times an infinity or a
// NaN is not: a row whose output is not finite is computed again from its visible
// keys alone, one warp per row (row_again).
//
// Warps: 0 issues TMA, 1 allocates TMEM and issues the products, 2 checks the starts,
// 4.. are the softmax and output warps, four per tile.
#include "attn_math.cuh"
#include "attn_prefill.h"
#include "common.cuh"
#include "kernels.h"
#include "tcgen05_ops.cuh"
#include "tensor_map.h"

namespace fp8moe {
using namespace sm100;
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kFew = 88, kMany = 208;
constexpr float kMove = 8.f;  // log2 of how far a score may exceed the reference

template <int D>
struct Shape {
  static constexpr int kTiles = D == 256 ? 1 : 2;  // of an item
  static constexpr int kKeys = D == 256 ? 64 : 128;
  static constexpr int kChunks = D / 64;           // boxes of 64 elements
  static constexpr int kQTile = 128 * D * 2, kSlot = kKeys * D * 2;
  static constexpr int kSlots = D == 64 ? 8 : 5;
  static constexpr int kThreads = 128 + 128 * kTiles;
  static constexpr size_t kSmem = (size_t)kTiles * kQTile + (size_t)kSlots * kSlot + 1024;
  static constexpr uint32_t kS = 0, kO = 2 * kKeys;  // TMEM columns: two S, then O of each tile
};

// Positions and rows fit 32 bits (Tq and Tk do); sums that may not are 64-bit.
template <int D>
struct Item {
  int q0, k0;        // first rows of the sequence
  int n, m;          // its queries and keys
  int tok0;          // the item's first token
  int kv, head0;     // key/value head, first query head
  int heads;         // of head0's on, that are the tile's own
  int lo[Shape<D>::kTiles], hi[Shape<D>::kTiles];  // blocks of each tile
  int first, last;   // blocks of all tiles
  bool any;          // tokens
};

__device__ __forceinline__ int clamp_start(const int32_t *starts, int b, int total) {
  const int v = __ldg(starts + b);
  return v < 0 ? 0 : v > total ? total : v;
}

// Item i: the items of a sequence's last tokens, which see most keys, come first.
// Sequence b owns the places [q_starts[b] / T + b, q_starts[b + 1] / T + b + 1) for
// its ceil(n / T) tiles of T tokens: found from the starts alone.
template <int D>
__device__ __forceinline__ Item<D> item_of(const PrefillArgs &p, int64_t i) {
  constexpr int kTiles = Shape<D>::kTiles, kKeys = Shape<D>::kKeys;
  Item<D> it;
  const int groups = p.n_kv * p.chunks, T = kTiles * p.tokens;
  const int group = (int)(i % groups), place = (int)(p.items / groups - 1 - i / groups);
  int b = 0;
  for (int end = p.B; end - b > 1;) {
    const int mid = (b + end) >> 1;
    if (clamp_start(p.q_starts, mid, p.Tq) / T + mid <= place) b = mid;
    else end = mid;
  }
  const int q0 = clamp_start(p.q_starts, b, p.Tq), q1 = clamp_start(p.q_starts, b + 1, p.Tq);
  const int k0 = clamp_start(p.k_starts, b, p.Tk), k1 = clamp_start(p.k_starts, b + 1, p.Tk);
  it.q0 = q0;
  it.k0 = k0;
  it.n = q1 > q0 ? q1 - q0 : 0;
  it.m = k1 > k0 ? k1 - k0 : 0;
  const int64_t tok0 = (int64_t)(place - (q0 / T + b)) * T;
  it.any = tok0 >= 0 && tok0 < it.n;
  it.tok0 = it.any ? (int)tok0 : 0;
  const int per_kv = p.n_heads / p.n_kv, chunk = group % p.chunks;
  it.kv = group / p.chunks;
  it.head0 = it.kv * per_kv + chunk * p.heads;
  it.heads = min(p.heads, per_kv - chunk * p.heads);
  it.first = it.last = 0;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int64_t a = (int64_t)it.tok0 + t * p.tokens;
    const int64_t e = min(a + p.tokens, (int64_t)it.n);
    it.lo[t] = it.hi[t] = 0;
    if (!it.any || a >= e) continue;
    // the keys that the tile's tokens see
    const int64_t off = (int64_t)it.m - it.n;
    int64_t hi = it.m, lo = 0;
    if (p.causal) hi = min(hi, e + off);
    if (p.window > 0) lo = max((int64_t)0, a + off - p.window + 1);
    if (lo >= hi) continue;
    it.lo[t] = (int)(lo / kKeys);
    it.hi[t] = (int)((hi + kKeys - 1) / kKeys);
    if (it.last == 0) it.first = it.lo[t];
    it.first = min(it.first, it.lo[t]);
    it.last = max(it.last, it.hi[t]);
  }
  return it;
}

// A row's score after the products: in units of log2, options applied.
__device__ __forceinline__ float option_score(float s, float scale, float cap, float slope, int back) {
  s *= scale;
  if (cap > 0.f) s = cap * tanh_f32(__fdividef(s, cap));
  return fmaf(slope, (float)back, s) * kLog2e;
}

// One row from its visible keys alone, by a warp: for rows that met values which are
// not finite.  32 keys at a time, a lane scoring one; then lane l adds up the
// elements l * D / 32 ... of their values.
template <int D>
__device__ __noinline__ void row_again(const PrefillArgs &p, const __nv_bfloat16 *q, const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                                       int lo, int hi, int pos, float slope, __nv_bfloat16 *out, float *lse) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int j0 = lo; j0 < hi; j0 += 32) {
    const int here = min(32, hi - j0);
    float s = -INFINITY;
    if (lane < here) {
      const __nv_bfloat16 *row = k + (int64_t)(j0 + lane) * p.k_stride;
      s = 0.f;
#pragma unroll 4
      for (int e = 0; e < D; e += 8) {
        const uint4 a = *reinterpret_cast<const uint4 *>(q + e), b = *reinterpret_cast<const uint4 *>(row + e);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s = fmaf(bf16_bits_to_float(u4_word(a, x) & 0xffffu), bf16_bits_to_float(u4_word(b, x) & 0xffffu), s);
          s = fmaf(__uint_as_float(u4_word(a, x) & 0xffff0000u), __uint_as_float(u4_word(b, x) & 0xffff0000u), s);
        }
      }
      s = option_score(s, p.scale, p.softcap, slope, j0 + lane - pos);
    }
    const float ref = fmaxf(m, warp_max(s));
    const float keep = m == ref ? 1.f : exp2_fast(m - ref), w = s == -INFINITY ? 0.f : exp2_fast(s - ref);
    m = ref;
    l = fmaf(l, keep, warp_sum(w));
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= keep;
    for (int j = 0; j < here; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const __nv_bfloat16 *row = v + (int64_t)(j0 + j) * p.v_stride + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(wj, __bfloat162float(row[e]), acc[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane * E + e] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[e] / l);
  if (lse != nullptr && lane == 0) *lse = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

__device__ __forceinline__ void give_up(volatile int *stop, int *err) {
  *stop = 1;
  set_error(err, DEV_ERR_TIMEOUT);
}

// Option: scores need more than a positive scale (a cap, slopes, another scale).
template <int D, bool Option>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1) prefill_kernel(const __grid_constant__ CUtensorMap tq,
                                                                       const __grid_constant__ CUtensorMap tk,
                                                                       const __grid_constant__ CUtensorMap tv, const PrefillArgs p) {
  using Z = Shape<D>;
  constexpr int kTiles = Z::kTiles, kKeys = Z::kKeys, kSlots = Z::kSlots;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full[kTiles], q_empty[kTiles], kv_full[kSlots], kv_empty[kSlots], s_full[2], p_full[2],
      o_full[kTiles];
  __shared__ uint32_t tmem_sh;
  __shared__ volatile int stop;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *ring = smem + kTiles * Z::kQTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < kTiles; ++t) mbar_init(&q_full[t], 1), mbar_init(&q_empty[t], 1), mbar_init(&o_full[t], 1);
    for (int s = 0; s < kSlots; ++s) mbar_init(&kv_full[s], 1), mbar_init(&kv_empty[s], 1);
    for (int b = 0; b < 2; ++b) mbar_init(&s_full[b], 1), mbar_init(&p_full[b], 4);
    stop = 0;
    fence_mbar_init();
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_sh, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_wait();
  pdl_trigger();

  // 384 threads start with 168 registers each; the eight softmax warps hold a row of
  // scores: 128 * 88 + 256 * 208 = 384 * 168 (checked against the build in ready_d).
  // (Each role's branch says so itself, which is where the compiler looks.)
  if (warp < 4) {
  if constexpr (kTiles == 2) fewer_registers<kFew>();
  if (warp == 0) {
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 0, q_phase = 0;  // a bit per tile
      const auto load = [&](const CUtensorMap *map, const Item<D> &it, int block) {
        if (!mbar_wait(&kv_empty[slot], phase ^ 1u, &stop, kWaitNs)) {
          give_up(&stop, p.err);
          return false;
        }
        mbar_arrive_expect_tx(&kv_full[slot], Z::kSlot);
#pragma unroll
        for (int c = 0; c < Z::kChunks; ++c)
          tma_load_3d(ring + (size_t)slot * Z::kSlot + c * (kKeys * 128), map, 64 * c, it.kv, it.k0 + block * kKeys,
                      &kv_full[slot]);
        if (++slot == kSlots) slot = 0, phase ^= 1u;
        return true;
      };
      bool ok = true;
      for (int64_t i = blockIdx.x; ok && i < p.items && !stop; i += gridDim.x) {
        const Item<D> it = item_of<D>(p, i);
        if (it.last == 0) continue;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (it.lo[t] >= it.hi[t]) continue;
          if (!mbar_wait(&q_empty[t], (q_phase >> t & 1u) ^ 1u, &stop, kWaitNs)) {
            give_up(&stop, p.err);
            ok = false;
            break;
          }
          q_phase ^= 1u << t;
          mbar_arrive_expect_tx(&q_full[t], (uint32_t)(p.tokens * p.heads * 128 * Z::kChunks));
#pragma unroll
          for (int c = 0; c < Z::kChunks; ++c)
            tma_load_3d(smem + t * Z::kQTile + c * (128 * 128), &tq, 64 * c, it.head0, it.q0 + it.tok0 + t * p.tokens,
                        &q_full[t]);
        }
        // in the order of their first use: keys one block ahead (with one tile, two)
        ok = ok && load(&tk, it, it.first);
        if (kTiles == 1 && it.first + 1 < it.last) ok = ok && load(&tk, it, it.first + 1);
        for (int j = it.first; ok && j < it.last; ++j) {
          ok = load(&tv, it, j);
          const int ahead = j + (kTiles == 1 ? 2 : 1);
          if (ok && ahead < it.last) ok = load(&tk, it, ahead);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t i_s = idesc_bf16(128, kKeys, false), i_o = idesc_bf16(128, D, true);
      int slot = 0, step = 0;  // step: of one tile's S buffers
      uint32_t phase = 0, q_phase = 0, p_phase = 0;
      bool ok = true;
      const auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok && !mbar_wait(bar, parity, &stop, kWaitNs)) {
          give_up(&stop, p.err);
          ok = false;
        }
        return ok;
      };
      // Descriptors differ from the first tile's and slot's in their start address
      // (16-byte units) alone; the asm keeps the compiler from holding all of them in
      // registers.
      const uint64_t q_desc = sw128_kmajor_desc(smem_u32(smem)), k_desc = sw128_kmajor_desc(smem_u32(ring)),
                     v_desc = sw128_rows_k_desc(smem_u32(ring), kKeys * 128);
      const auto scores = [&](int t, int buf, int s) {  // S[buf] = Q[t] K[slot s]^T
        uint64_t a = q_desc + (uint64_t)(t * (Z::kQTile / 16)), b = k_desc + (uint64_t)(s * (Z::kSlot / 16));
        asm volatile("" : "+l"(a), "+l"(b));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_bf16_ss(tmem + Z::kS + buf * kKeys, a + ((k >> 2) * (128 * 128) + (k & 3) * 32) / 16,
                      b + ((k >> 2) * (kKeys * 128) + (k & 3) * 32) / 16, i_s, k > 0 ? 1u : 0u);
        mma_commit(&s_full[buf]);
      };
      const auto values = [&](int t, int buf, int s, bool more) {  // O[t] (+)= P[buf] V[slot s]
        uint64_t b = v_desc + (uint64_t)(s * (Z::kSlot / 16));
        asm volatile("" : "+l"(b));
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_bf16_ts(tmem + Z::kO + t * D, tmem + Z::kS + buf * kKeys + k * 8, b + k * (2048 / 16), i_o, more || k > 0 ? 1u : 0u);
        mma_commit(&o_full[t]);
      };
      const auto advance = [&] {
        mma_commit(&kv_empty[slot]);
        if (++slot == kSlots) slot = 0, phase ^= 1u;
      };
      for (int64_t i = blockIdx.x; ok && i < p.items && !stop; i += gridDim.x) {
        const Item<D> it = item_of<D>(p, i);
        if (it.last == 0) continue;
        if constexpr (kTiles == 2) {
          // block j of the keys has a slot, and is used by both tiles; values likewise
          if (!wait(&kv_full[slot], phase)) break;
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (it.lo[t] < it.hi[t] && it.lo[t] == it.first) {
              if (!wait(&q_full[t], q_phase >> t & 1u)) break;
              q_phase ^= 1u << t;
              tc_fence_after();
              scores(t, t, slot);
              if (it.hi[t] == it.first + 1) mma_commit(&q_empty[t]);
            }
          if (!ok) break;
          advance();
          for (int j = it.first; ok && j < it.last; ++j) {
            const int v_slot = slot;
            if (!wait(&kv_full[slot], phase)) break;
            if (++slot == kSlots) slot = 0, phase ^= 1u;
            if (j + 1 < it.last && !wait(&kv_full[slot], phase)) break;
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (it.lo[t] <= j && j < it.hi[t]) {
                if (!wait(&p_full[t], p_phase >> t & 1u)) break;
                p_phase ^= 1u << t;
                tc_fence_after();
                values(t, t, v_slot, j > it.lo[t]);
              }
              if (it.lo[t] <= j + 1 && j + 1 < it.hi[t]) {
                if (j + 1 == it.lo[t]) {
                  if (!wait(&q_full[t], q_phase >> t & 1u)) break;
                  q_phase ^= 1u << t;
                  tc_fence_after();
                }
                scores(t, t, slot);
                if (it.hi[t] == j + 2) mma_commit(&q_empty[t]);
              }
            }
            if (!ok) break;
            mma_commit(&kv_empty[v_slot]);
            if (j + 1 < it.last) advance();
          }
        } else {
          if (!wait(&q_full[0], q_phase)) break;
          q_phase ^= 1u;
          for (int j = it.first; ok && j < it.last && j < it.first + 2; ++j) {
            if (!wait(&kv_full[slot], phase)) break;
            tc_fence_after();
            scores(0, (step + j - it.first) & 1, slot);
            if (j + 1 == it.last) mma_commit(&q_empty[0]);
            advance();
          }
          for (int j = it.first; ok && j < it.last; ++j, ++step) {
            const int buf = step & 1;
            if (!wait(&kv_full[slot], phase) || !wait(&p_full[buf], p_phase >> buf & 1u)) break;
            p_phase ^= 1u << buf;
            tc_fence_after();
            values(0, buf, slot, j > it.first);
            advance();
            if (j + 2 < it.last) {
              if (!wait(&kv_full[slot], phase)) break;
              tc_fence_after();
              scores(0, buf, slot);
              if (j + 3 == it.last) mma_commit(&q_empty[0]);
              advance();
            }
          }
        }
      }
    }
  } else if (warp == 2 && blockIdx.x == 0) {
    bool bad = false;
    for (int b = lane; b <= p.B; b += 32) {
      const int qs = __ldg(p.q_starts + b), ks = __ldg(p.k_starts + b);
      bad |= qs < 0 || qs > p.Tq || ks < 0 || ks > p.Tk;
      if (b < p.B) bad |= __ldg(p.q_starts + b + 1) < qs || __ldg(p.k_starts + b + 1) < ks;
    }
    if (bad) set_error(p.err, DEV_ERR_BOUNDS);
  }
  } else {
    if constexpr (kTiles == 2) more_registers<kMany>();
    const int t = (warp - 4) >> 2;  // tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int row = (warp & 3) * 32 + lane;  // of the tile
    const uint32_t t_o = tmem + lanes + Z::kO + t * D;
    const int r_tok = row / p.heads, r_head = row - r_tok * p.heads;
    const float scale2 = Option ? 1.f : p.scale * kLog2e;
    int step = 0;               // S buffers used (one tile)
    uint32_t s_phase = 0, o_count = 0;  // products with V that the tile has had
    bool ok = true;
    for (int64_t i = blockIdx.x; ok && i < p.items; i += gridDim.x) {
      const Item<D> it = item_of<D>(p, i);
      if (!it.any) continue;
      // of the sequence (past its end: a row of no use); a row's position is below the
      // last key's by the tokens that follow it
      const uint32_t tok = (uint32_t)(it.tok0 + t * p.tokens) + (uint32_t)r_tok;
      const bool mine = r_tok < p.tokens && r_head < it.heads && tok < (uint32_t)it.n;
      const int pos = it.m - (int)((uint32_t)it.n - tok);
      // the keys that this row sees, and those that all of the tile's rows do
      int see_lo = 0, see_hi = it.m, all_lo = 0, all_hi = it.m;
      if (p.causal) {
        see_hi = max(0, min(it.m, pos + 1));
        all_hi = max(0, min(it.m, it.m - (it.n - (it.tok0 + t * p.tokens)) + 1));
      }
      if (p.window > 0) {
        const int behind = it.n - it.tok0 - (t + 1) * p.tokens;  // tokens after the tile's
        see_lo = (int)max(INT64_C(0), min((int64_t)it.m, (int64_t)pos - p.window + 1));
        all_lo = (int)max(INT64_C(0), (int64_t)it.m - max(behind, 0) - p.window);
      }
      const float slope = Option && p.slopes != nullptr && mine ? __ldg(p.slopes + it.head0 + r_head) : 0.f;
      float ref = -INFINITY;
      uint64_t sum2 = 0;
      const int lo = it.lo[t], hi = it.hi[t];
      for (int j = lo; j < hi; ++j) {
        const int buf = kTiles == 2 ? t : step & 1;
        if (!mbar_wait(&s_full[buf], s_phase >> buf & 1u, &stop, kWaitNs)) {
          give_up(&stop, p.err);
          ok = false;
          break;
        }
        s_phase ^= 1u << buf;
        tc_fence_after();
        const uint32_t t_s = tmem + lanes + Z::kS + buf * kKeys;
        uint32_t s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(t_s + c, s + c);
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_wait_ld(s + c);
        const int key0 = j * kKeys;
        if constexpr (Option) {
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            s[c] = __float_as_uint(option_score(__uint_as_float(s[c]), p.scale, p.softcap, slope, key0 + c - pos));
        }
        if (key0 < all_lo || key0 + kKeys > all_hi) {
          const int from = see_lo - key0, to = see_hi - key0;
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (c < from || c >= to) s[c] = __float_as_uint(-INFINITY);
        }
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) top[c] = __uint_as_float(s[c]);
#pragma unroll
        for (int c = 4; c < kKeys; ++c) top[c & 3] = fmaxf(top[c & 3], __uint_as_float(s[c]));
        const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale2;
        const bool move = most > ref + kMove;
        if (__any_sync(0xffffffffu, move)) {
          const float keep = !move ? 1.f : ref == -INFINITY ? 0.f : exp2_fast(ref - most);
          if (move) ref = most;
          const uint64_t kk = pack_f32x2(keep, keep);
          sum2 = mul_f32x2(sum2, kk);
          if (j > lo) {
            // S of this block is ready, so the products with V up to the one before
            // last are done (with two tiles the last too)
            if (kTiles == 1 && !mbar_wait(&o_full[t], (o_count - 1u) & 1u, &stop, kWaitNs)) {
              give_up(&stop, p.err);
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(t_o + c, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * keep);
              tmem_st32(t_o + c, o);
            }
          }
        }
        const float minus = ref == -INFINITY ? 0.f : -ref;
        const uint64_t mul = pack_f32x2(scale2, scale2), add = pack_f32x2(minus, minus);
        uint64_t part = 0;
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const float2 f = unpack_f32x2(
                fma_f32x2(pack_f32x2(__uint_as_float(s[c + x]), __uint_as_float(s[c + x + 1])), mul, add));
            const float p0 = exp2_fast(f.x), p1 = exp2_fast(f.y);
            part = add_f32x2(part, pack_f32x2(p0, p1));
            w[x / 2] = bf16x2_of(p0, p1);
          }
          tmem_st16(t_s + c / 2, w);
        }
        sum2 = add_f32x2(sum2, part);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
        ++step;
        ++o_count;
      }
      if (!ok) break;
      const float2 sums = unpack_f32x2(sum2);
      const float sum = sums.x + sums.y;
      const float inv = sum > 0.f || !(sum == sum) ? 1.f / sum : 0.f;
      if (lo < hi) {
        if (!mbar_wait(&o_full[t], (o_count - 1u) & 1u, &stop, kWaitNs)) {
          give_up(&stop, p.err);
          break;
        }
        tc_fence_after();
      }
      __nv_bfloat16 *out = p.out + (it.q0 + (int64_t)tok) * p.out_stride + (int64_t)(it.head0 + r_head) * D;
      bool odd = false;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (lo < hi) {
          tmem_ld32(t_o + c, o);
          tmem_wait_ld(o);
        }
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          const float f = inv == 0.f ? 0.f : __uint_as_float(o[x]) * inv, g = inv == 0.f ? 0.f : __uint_as_float(o[x + 1]) * inv;
          odd |= !(fabsf(f) <= 3.402823466e38f && fabsf(g) <= 3.402823466e38f);
          o[x / 2] = bf16x2_of(f, g);
        }
        if (mine) {
#pragma unroll
          for (int x = 0; x < 16; x += 4) *reinterpret_cast<uint4 *>(out + c + 2 * x) = make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
        }
      }
      if (mine && p.lse != nullptr)
        p.lse[(it.q0 + (int64_t)tok) * p.n_heads + it.head0 + r_head] = inv == 0.f ? -INFINITY : kLn2 * (ref + log2f(sum));
      __syncwarp();
      for (uint32_t left = __ballot_sync(0xffffffffu, odd && mine); left != 0; left &= left - 1) {
        const int from = __ffs(left) - 1;
        const int64_t r = it.q0 + (int64_t)__shfl_sync(0xffffffffu, tok, from);
        const int at = __shfl_sync(0xffffffffu, pos, from);
        const int head = it.head0 + __shfl_sync(0xffffffffu, r_head, from);
        const int l = __shfl_sync(0xffffffffu, see_lo, from), h = __shfl_sync(0xffffffffu, see_hi, from);
        row_again<D>(p, p.q + r * p.q_stride + (int64_t)head * D, p.k + (int64_t)it.k0 * p.k_stride + (int64_t)it.kv * D,
                     p.v + (int64_t)it.k0 * p.v_stride + (int64_t)it.kv * D, l, h, at, __shfl_sync(0xffffffffu, slope, from),
                     p.out + r * p.out_stride + (int64_t)head * D, p.lse == nullptr ? nullptr : p.lse + r * p.n_heads + head);
      }
    }
  }
  __syncthreads();
  if (stop) {
    // copies and products in flight land before the memory goes away
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 50000ull) {
    }
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

bool map_rows(CUtensorMap *m, const void *p, int d, int heads, int64_t rows, int64_t stride, int box_heads, int box_rows) {
  const uint64_t sizes[3] = {(uint64_t)d, (uint64_t)heads, (uint64_t)rows}, strides[2] = {(uint64_t)d * 2, (uint64_t)stride * 2};
  const uint32_t box[3] = {64, (uint32_t)box_heads, (uint32_t)box_rows};
  return encode_tile_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, sizes, strides, box);
}

template <int D>
cudaError_t launch_d(const PrefillArgs &a, int sms, cudaStream_t s) {
  using Z = Shape<D>;
  CUtensorMap tq, tk, tv;
  // without keys nothing of k and v is read
  const bool keys = a.Tk > 0;
  if (!map_rows(&tq, a.q, D, a.n_heads, a.Tq, a.q_stride, a.heads, a.tokens) ||
      !map_rows(&tk, keys ? a.k : a.q, D, keys ? a.n_kv : 1, keys ? a.Tk : 1, keys ? a.k_stride : a.q_stride, 1, Z::kKeys) ||
      !map_rows(&tv, keys ? a.v : a.q, D, keys ? a.n_kv : 1, keys ? a.Tk : 1, keys ? a.v_stride : a.q_stride, 1, Z::kKeys))
    return cudaErrorInvalidValue;
  const bool option = a.softcap > 0.f || a.slopes != nullptr || !(a.scale > 0.f);
  return launch_pdl(option ? prefill_kernel<D, true> : prefill_kernel<D, false>, dim3((unsigned)(a.items < sms ? a.items : sms)),
                    dim3(Z::kThreads), Z::kSmem, s, tq, tk, tv, a);
}

template <int D>
cudaError_t ready_d() {
  for (auto k : {prefill_kernel<D, true>, prefill_kernel<D, false>}) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<D>::kSmem);
    if (e != cudaSuccess) return e;
    // the softmax warps would wait forever for registers that the launch does not have
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, k);
    if (e != cudaSuccess) return e;
    if (Shape<D>::kTiles == 2 && at.numRegs * 3 < kFew + 2 * kMany) return cudaErrorInvalidKernelImage;
  }
  return cudaSuccess;
}

}  // namespace

void plan_prefill(PrefillArgs *a, int d) {
  // pieces of at most 16 heads, as even as may be
  const int per_kv = a->n_heads / a->n_kv;
  a->chunks = (per_kv + 15) / 16;
  a->heads = (per_kv + a->chunks - 1) / a->chunks;
  a->tokens = 128 / a->heads;
  const int T = a->tokens * (d == 256 ? 1 : 2);
  a->items = ((int64_t)a->Tq / T + a->B) * a->n_kv * a->chunks;
}

cudaError_t ready_prefill(int d) { return d == 64 ? ready_d<64>() : d == 128 ? ready_d<128>() : ready_d<256>(); }

cudaError_t launch_prefill(const PrefillArgs &a, int d, int sms, cudaStream_t s) {
  return d == 64 ? launch_d<64>(a, sms, s) : d == 128 ? launch_d<128>(a, sms, s) : launch_d<256>(a, sms, s);
}

}  // namespace fp8moe
