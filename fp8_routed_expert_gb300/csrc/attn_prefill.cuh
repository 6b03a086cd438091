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
//   P = exp2(S * scale - ref)    in registers: one thread per row, no shuffles; back to
//                 TMEM as bf16 over S
//   O += P V      tcgen05.mma with P from TMEM; V as it lies (rows along K)
// The two tiles (or, with one tile, two S buffers of neighbouring blocks) alternate:
// one is in its softmax while the other's products run.  So a block's softmax has to
// take no longer than the other's products, about 1300 cycles, and while these read
// their operands shared memory has no bandwidth left: a row is one thread's, which
// keeps all it needs in registers and reads its scores once, 32 at a time.  (Two threads
// per row that exchanged their largest scores, or registers that spilled, took two to
// three times as long.)  Nothing waits for the row's largest score either: the softmax
// reference is of the blocks before.  Where the largest so far exceeds it by 2^8 it
// moves there, and only then is O read, scaled and written back.  A weight may so exceed
// 2^8 for a block, which f32 sums and bf16 weights hold as exactly as one below 1; where
// one leaves f32's range (scores that rise by 88 within a block) the row is computed
// again (below).  Rows that have no reference yet take it from the block itself, which is
// then read twice.  With slopes, which lower the scores of far keys, blocks go from the
// last to the first: the first reference is then the largest (forwards it moves, and O is
// rewritten, in every block: 8192 tokens, 16 heads of 128 elements, 305 us, so 245 at that step).
// Without them forwards is 3% faster, as an item's two tiles start together.
//
// What bounds it: 16384 tokens, 32 heads over 8 of 128 elements, take 1355 to 1415 us in
// bursts of a few milliseconds, 1560 to 1620 TFLOP/s or 81 to 85% of the measured bf16 rate
// of a burst, and 1450 back to back, 89% of the sustained rate; a warp's softmax of a block
// and the other tile's products take about the same time.  8192 tokens, 16 heads over 8:
// 1460 TFLOP/s, with 256 elements 1370 (one tile), with 64 885 (the exponentials are twice
// as many per product).  12 prompts of up to 2048 in 110 us: the tensor cores are busy 45%
// of it, as masked blocks cost twice, and an item has few of them to spread its first and
// last steps over; 60 of up to 700 with slopes 102.  The few registers that some kernels
// spill are an item's, not a block's (5 local loads per warp and item, 0.1% of the
// instructions); those of shared items without options take 8 per warp and block, 1.3%.
//
// Weights are rounded to bf16 for the second product, the matrix unit's type for bf16
// values: 2^-8 of each weight at most.  lse is of the f32 weights' sum; the outputs are
// divided by one that takes the heaviest weight of each block as it was rounded, so that a
// key with all of the weight gives its value to the bit.  Against 64 bits the outputs of 12
// prompts are off by 0.00206 of their size; the outputs' own rounding is 0.0016 of it.  (The
// sum of all rounded weights: 0.00204, for 7 to 27% of the time, 16384 tokens 1375 us, so
// 1485, 60 prompts with slopes 99.6 and 126.)
// A caller may choose 16 bits (Terms = 2): what a weight's first 8 bits leave is the A
// operand of a second product, half as many products again, and of each weight 2^-15 is
// lost at most, the outputs off by 0.0016.  us, 8 and 16 bits: 12 prompts 109 and 148, 16384
// tokens 1360 and 2015, capped chunks 138 and 175, 60 prompts with slopes 102 and 133.
//
// Blocks that no row sees are not visited; masks are applied in blocks that not all
// rows see in full.  A hidden value's weight is zero, but zero times an infinity or a
// NaN is not: a row whose output is not finite is computed again from its visible
// keys alone, one warp per row (row_again), which is slow but bounded (the
// limit of the other roles' waits counts on it).
//
// A launch has a block per item, the longest first; a running one asks for the next
// item that has not started (cluster launch control), so no counter in memory is
// needed and the last items are short.  Where a call has so few items that whole clusters
// of CTAs are resident for each, a cluster shares an item's blocks and joins the parts
// through distributed shared memory (plan_prefill, Parts).
//
// Warps: 0 issues TMA, 1 allocates TMEM and issues the products, 2 asks for items, 4..
// are the softmax and output warps, four per tile.
#pragma once

#include "attn_math.cuh"
#include "attn_prefill.h"
#include "common.cuh"
#include "kernels.h"
#include "tcgen05_ops.cuh"
#include "tensor_map.h"

namespace fp8moe {
using namespace sm100;
namespace {

// A wait's limit: two seconds, and what a warp's 32 rows take where they are computed
// again (row_again), 5 us for each key, four times over: the other roles wait meanwhile.
constexpr uint64_t kWaitNs = 2000000000ull, kWaitNsPerKey = 20000ull;
constexpr int kStage = 32 * 128;  // bytes in which a warp turns 64 columns of its 32 rows of outputs
constexpr float kMove = 8.f;  // log2 of how far a score may exceed the reference

template <int D>
struct Shape {
  static constexpr int kTiles = D == 256 ? 1 : 2;  // of an item
  static constexpr int kKeys = D == 256 ? 64 : 128;
  static constexpr int kChunks = D / 64;           // boxes of 64 elements
  static constexpr int kQTile = 128 * D * 2, kSlot = kKeys * D * 2;
  static constexpr int kSlots = D == 64 ? 8 : 4;
  static constexpr int kThreads = 128 + 128 * kTiles;
  static constexpr uint32_t kS = 0, kO = 2 * kKeys;  // TMEM columns: two S, then O of each tile
};

// Positions and rows fit 32 bits (Tq and Tk do); sums that may not are 64-bit.
struct Item {
  int q0, k0;      // first rows of the sequence
  int n, m;        // its queries and keys; n = 0: no more items
  int tok0;        // the item's first token
  int kv, head0;   // key/value head, first query head
  int heads;       // of head0's on, that are the tile's own
  int block0;                    // turn j takes block block0 + j (with slopes block0 - j)
  int lo[2], hi[2];              // turns whose block each tile's tokens see some keys of
  int whole_lo[2], whole_hi[2];  // and those whose block all of them see all of
  int first, last;               // turns of all tiles
};

constexpr int kAhead = 2;  // items asked for ahead

template <int D>
struct Control {
  static constexpr int kTiles = Shape<D>::kTiles, kSlots = Shape<D>::kSlots;
  uint8_t answer[16];
  Item items[kAhead];
  uint64_t q_full[kTiles], q_empty[kTiles], kv_full[kSlots], kv_empty[kSlots], s_full[2], p_full[2], o_full[2], answered,
      item_full[kAhead], item_empty[kAhead];
  uint32_t tmem, odd[4];  // odd: rows of this CTA's share whose output is not finite
  int stop;
};
template <int D>
constexpr size_t smem_bytes() {
  return (size_t)Shape<D>::kTiles * (Shape<D>::kQTile + 4 * kStage) + (size_t)Shape<D>::kSlots * Shape<D>::kSlot + sizeof(Control<D>);
}

__device__ __forceinline__ int clamp_start(const int32_t *starts, int b, int total) {
  const int v = __ldg(starts + b);
  return v < 0 ? 0 : v > total ? total : v;
}

// The tokens of an item.
template <int D>
__device__ __forceinline__ int item_tokens(const PrefillArgs &p) {
  return Shape<D>::kTiles * p.tokens;
}

// Where the r-th piece of T tokens lies, the longest first: those at the end of a
// sequence see most keys, so pieces go by their number within the sequence, the largest
// first, then by sequence.  Up to 32 * kHeld sequences, of which each lane holds kHeld
// pieces' counts; -1: no such piece.  For the whole warp.
constexpr int kHeld = 4;
struct Piece {
  int b, index;
};
__device__ __forceinline__ Piece piece_of(const int (&counts)[kHeld], int r) {
  const int lane = threadIdx.x & 31;
  const auto from = [&](int level) {  // pieces of that number and above
    int n = 0;
#pragma unroll
    for (int u = 0; u < kHeld; ++u) n += max(0, counts[u] - level);
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
  };
  int most = 0;
#pragma unroll
  for (int u = 0; u < kHeld; ++u) most = max(most, counts[u]);
  int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);
  if (r >= from(0)) return Piece{-1, 0};
  while (hi - lo > 1) {  // from(lo) > r >= from(hi)
    const int mid = (lo + hi) >> 1;
    if (from(mid) > r) lo = mid;
    else hi = mid;
  }
  int k = r - from(lo + 1), b = -1;  // the k-th sequence with more than lo pieces
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const uint32_t have = __ballot_sync(0xffffffffu, counts[u] > lo);
    const int n = __popc(have);
    if (b < 0 && k < n) {
      const bool mine = (have >> lane & 1u) && __popc(have & ((1u << lane) - 1u)) == k;
      b = 32 * u + __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    }
    k -= n;
  }
  return Piece{b, lo};
}
// The same for any number of sequences, in the order of their rows from the last on:
// sequence b owns the places [q_starts[b] / T + b, q_starts[b + 1] / T + b + 1) for its
// ceil(n / T) pieces, found from the starts alone.
__device__ __forceinline__ Piece piece_at(const PrefillArgs &p, int place, int T) {
  int b = 0;
  for (int end = p.B; end - b > 1;) {
    const int mid = (b + end) >> 1;
    if (clamp_start(p.q_starts, mid, p.Tq) / T + mid <= place) b = mid;
    else end = mid;
  }
  return Piece{b, place - (clamp_start(p.q_starts, b, p.Tq) / T + b)};
}

// Piece `index` of sequence b, and a group of heads; false if it has no tokens.  Of an
// item that is split, the turns of CTA `rank`.
template <int D, bool Split>
__device__ __forceinline__ bool item_of(const PrefillArgs &p, int b, int index, int group, int rank, Item *it) {
  constexpr int kTiles = Shape<D>::kTiles, kKeys = Shape<D>::kKeys;
  const int q0 = clamp_start(p.q_starts, b, p.Tq), q1 = clamp_start(p.q_starts, b + 1, p.Tq);
  const int k0 = clamp_start(p.k_starts, b, p.Tk), k1 = clamp_start(p.k_starts, b + 1, p.Tk);
  const int n = q1 - q0, m = max(k1 - k0, 0);
  const int64_t tok0 = (int64_t)index * item_tokens<D>(p);
  if (tok0 < 0 || tok0 >= n) return false;
  it->q0 = q0;
  it->k0 = k0;
  it->n = n;
  it->m = m;
  it->tok0 = (int)tok0;
  const int per_kv = p.n_heads / p.n_kv, chunk = group % p.chunks;
  it->kv = group / p.chunks;
  it->head0 = it->kv * per_kv + chunk * p.heads;
  it->heads = min(p.heads, per_kv - chunk * p.heads);
  int first = 0, last = 0;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    // the tile's tokens [a, e), and the keys that some and that all of them see
    const int64_t a = tok0 + t * p.tokens, e = min(a + p.tokens, (int64_t)n), off = (int64_t)m - n;
    int64_t hi = m, lo = 0, all_hi = m, all_lo = 0;
    if (p.causal) hi = min(hi, e + off), all_hi = min(all_hi, a + off + 1);
    if (p.window > 0) lo = max(lo, a + off - p.window + 1), all_lo = max(all_lo, e + off - p.window);
    const bool some = a < e && lo < hi;
    it->lo[t] = some ? (int)(lo / kKeys) : 0;  // blocks, as yet
    it->hi[t] = some ? (int)((hi + kKeys - 1) / kKeys) : 0;
    it->whole_lo[t] = (int)((all_lo + kKeys - 1) / kKeys);
    it->whole_hi[t] = all_hi > 0 ? (int)(all_hi / kKeys) : 0;
    if (some) {
      first = last == 0 ? it->lo[t] : min(first, it->lo[t]);
      last = max(last, it->hi[t]);
    }
  }
  it->first = 0;
  it->last = last - first;
  it->block0 = p.slopes == nullptr ? first : last - 1;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int lo = it->lo[t], hi = it->hi[t], whole_lo = it->whole_lo[t], whole_hi = it->whole_hi[t];
    if (p.slopes == nullptr) {
      it->lo[t] = lo - first, it->hi[t] = hi - first;
      it->whole_lo[t] = whole_lo - first, it->whole_hi[t] = whole_hi - first;
    } else {
      it->lo[t] = last - hi, it->hi[t] = last - lo;
      it->whole_lo[t] = last - whole_hi, it->whole_hi[t] = last - whole_lo;
    }
  }
  if constexpr (Split) {  // this CTA's turns
    const int64_t turns = it->last;
    it->first = (int)(turns * rank / p.splits);
    it->last = (int)(turns * (rank + 1) / p.splits);
    if (it->first == it->last) it->first = it->last = 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) it->lo[t] = max(it->lo[t], it->first), it->hi[t] = min(it->hi[t], it->last);
  }
  return true;
}

// A row's score after the products: in units of log2, options applied.
__device__ __forceinline__ float option_score(float s, float scale, float cap, float slope, int back) {
  s *= scale;
  if (cap > 0.f) s = cap * tanh_f32(s / cap);
  return fmaf(slope, (float)back, s) * kLog2e;
}

// Caps up to here: cap tanh(y) = cap - 2 cap / (1 + e^2y).  The quotient is off by seven
// halves of a step or less (its sum with 1, four products, a reciprocal of two) and what
// the power of two adds, and the constants and the difference by a few more: 2^-19 of the
// cap, which at 128 is 2.4e-4 of a score.  Above it tanh itself, whose error goes with the
// score, 2^-20 of it.  (8192 tokens, 16/8 heads of 64, 128 and 256 elements, a cap of 400:
// 386, 410 and 468 us, with the cap's way 334, 359 and 443.)
constexpr float kUsualCap = 128.f;

// 1 / (1 + 2^(s * unit)) of 32 scores, unit = 2 log2(e) scale / cap; or tanh(s * unit), unit =
// scale / cap.  Four scores share a reciprocal (of a product below 2^121: from 2^30 on the
// fraction no longer tells from zero): 8192 tokens, 16/8 heads of 64, 128 and 256
// elements, 340, 362 and 438 us; two to a reciprocal 373, 373 and 462, one each 360, 369
// and 531.  tanh without its polynomial: 693, 717 and 1078.  A NaN so reaches three
// neighbours; the row is computed again in any case.
template <bool Usual>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[32], float unit) {
  if constexpr (!Usual) {
    // Where all 32 are below 0.6, which nearly all are under so high a cap, by the
    // polynomial, two at a time; else the warp takes tanh_f32's both ways.
    float most = 0.f;
#pragma unroll
    for (int c = 0; c < 32; c += 2) most = max3(most, fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
    if (__all_sync(0xffffffffu, most * fabsf(unit) < 0.6f)) {
      const uint64_t u2 = pack_f32x2(unit, unit);
      const auto both = [](float f) { return pack_f32x2(f, f); };
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const uint64_t y = mul_f32x2(pack_f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), u2), z = mul_f32x2(y, y);
        uint64_t t = fma_f32x2(z, both(kTanh[4]), both(kTanh[3]));
        t = fma_f32x2(z, t, both(kTanh[2]));
        t = fma_f32x2(z, t, both(kTanh[1]));
        t = fma_f32x2(z, t, both(kTanh[0]));
        const float2 f = unpack_f32x2(fma_f32x2(mul_f32x2(y, z), t, y));
        s[c] = __float_as_uint(f.x), s[c + 1] = __float_as_uint(f.y);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) s[c] = __float_as_uint(tanh_f32(__uint_as_float(s[c]) * unit));
    }
    return;
  }
  const uint64_t u2 = pack_f32x2(unit, unit), one = pack_f32x2(1.f, 1.f);
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    const auto power = [&](int k) {
      const float2 x = unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), u2));
      return add_f32x2(pack_f32x2(exp2_fast(min_nan(x.x, 30.f)), exp2_fast(min_nan(x.y, 30.f))), one);
    };
    const uint64_t f = power(c), g = power(c + 2), fg = mul_f32x2(f, g);
    const float2 q = unpack_f32x2(fg);
    const float r = rcp_fast(q.x * q.y);
    const uint64_t t = mul_f32x2(pack_f32x2(q.y, q.x), pack_f32x2(r, r));
    const float2 a = unpack_f32x2(mul_f32x2(t, g)), b = unpack_f32x2(mul_f32x2(t, f));
    s[c] = __float_as_uint(a.x), s[c + 1] = __float_as_uint(a.y), s[c + 2] = __float_as_uint(b.x), s[c + 3] = __float_as_uint(b.y);
  }
}

// One row from its visible keys alone, by a warp: for rows that met values which are
// not finite.  32 keys at a time, a lane scoring one; then lane l adds up the
// elements l * D / 32 ... of their values, sixteen keys on their way.  Two to five us for 32
// keys, a hundred times what they take in a tile: 4096 tokens, 8 heads of 128 elements, whose
// first value is a NaN 13.4 ms instead of 0.12 (18.8 with a key at a time).
template <int D>
__device__ __noinline__ void row_again(const PrefillArgs &p, const __nv_bfloat16 *q, const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                                       int lo, int hi, int pos, float slope, __nv_bfloat16 *out, float *lse) {
  constexpr int E = D / 32, kAtOnce = 16;
  struct alignas(2 * E) Part {
    uint32_t two[E / 2];
  };
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
#pragma unroll 8
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
    const __nv_bfloat16 *first = v + (int64_t)j0 * p.v_stride + lane * E;
#pragma unroll 1
    for (int j = 0; j < here; j += kAtOnce) {
      Part x[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) x[u] = *reinterpret_cast<const Part *>(first + (int64_t)min(j + u, here - 1) * p.v_stride);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const float wj = __shfl_sync(0xffffffffu, w, j + u);
        if (j + u < here) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            acc[e] = fmaf(wj, e % 2 == 0 ? bf16_bits_to_float(x[u].two[e / 2] & 0xffffu) : __uint_as_float(x[u].two[e / 2] & 0xffff0000u), acc[e]);
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane * E + e] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[e] / l);
  if (lse != nullptr && lane == 0) *lse = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

// An item that a cluster's CTAs have split (few items): its rows are shared out, `held`
// neighbouring ones to a CTA, and each CTA pushes its part of a row, the output of its
// keys alone and (reference, log2 of the sum), to the row's CTA: [rank][row % held] over
// the slots of keys and values and over the queries, which nobody needs any longer.
struct PartStats {
  float ref, log;  // kNoPart: the part has no blocks, and its output is not there
};
constexpr float kNoPart = -3e38f;
struct Parts {
  int rows, held;  // held * splits is a tile's or two tiles' rows at most: splits is a power of two
  template <int D>
  __device__ __forceinline__ static Parts of(const PrefillArgs &p, int n, int tok0) {
    static_assert(Shape<D>::kTiles * 128 * D * 4 <= Shape<D>::kSlots * Shape<D>::kSlot, "parts fit");
    const int rows = min(item_tokens<D>(p), n - tok0) * p.heads;
    return Parts{rows, (rows + p.splits - 1) / p.splits};
  }
};

__device__ __forceinline__ void give_up(volatile int *stop, int *err) {
  *stop = 1;
  set_error(err, DEV_ERR_TIMEOUT);
}

// The rows of this CTA's share from the cluster's parts; by all its threads.
template <int D>
__device__ __noinline__ void join_parts(const PrefillArgs &p, Control<D> &ctl, uint8_t *smem, uint8_t *ring, int rank) {
  const Item &it = ctl.items[0];
  const Parts parts = Parts::of<D>(p, it.n, it.tok0);
  const auto used = [&](int r) { return r < parts.rows && r % p.heads < it.heads; };
  // A thread per 8 elements of a row: the part that adds most to the sum counts as one.
  for (int u = threadIdx.x; u < parts.held * (D / 8); u += Shape<D>::kThreads) {
    const int place = u / (D / 8), e = u % (D / 8) * 8, r = rank * parts.held + place;
    if (!used(r)) continue;
    const PartStats *stats = reinterpret_cast<const PartStats *>(smem) + place;
    const float *o = reinterpret_cast<const float *>(ring) + place * D + e;
    PartStats best = {-INFINITY, 0.f};
#pragma unroll 4
    for (int c = 0; c < p.splits; ++c) {
      const PartStats s = stats[c * parts.held];
      if (s.ref + s.log > best.ref + best.log) best = s;
    }
    const bool none = best.ref == -INFINITY;  // (where a part has no blocks too)
    float acc[8] = {}, total = 0.f, odd = 0.f;
#pragma unroll 2
    for (int c = 0; c < p.splits; ++c) {
      const PartStats s = stats[c * parts.held];
      if (s.log == kNoPart) continue;
      const float w = none ? 0.f : exp2_fast((s.ref - best.ref) + (s.log - best.log));
      total += w;
      const float4 f = *reinterpret_cast<const float4 *>(o + c * parts.held * D), g = *reinterpret_cast<const float4 *>(o + c * parts.held * D + 4);
      const float v[8] = {f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w};
      if (!(s.log < 200.f)) odd = NAN;  // the sum is not finite
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        odd = fmaf(v[x], 0.f, odd);  // (of a part whose keys all weigh nothing too)
        acc[x] = fmaf(v[x], w, acc[x]);
      }
    }
    const float inv = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      acc[x] *= inv;
      odd = fmaf(acc[x], 0.f, odd);
    }
    if (!(odd == 0.f)) atomicOr(&ctl.odd[place / 32], 1u << (place % 32));
    const int64_t at = it.q0 + (int64_t)it.tok0 + r / p.heads;
    const int h = it.head0 + r % p.heads;
    *reinterpret_cast<uint4 *>(p.out + at * p.out_stride + (int64_t)h * D + e) =
        make_uint4(bf16x2_of(acc[0], acc[1]), bf16x2_of(acc[2], acc[3]), bf16x2_of(acc[4], acc[5]), bf16x2_of(acc[6], acc[7]));
    if (e == 0 && p.lse != nullptr) p.lse[at * p.n_heads + h] = total > 0.f ? kLn2 * (best.ref + (best.log + log2f(total))) : -INFINITY;
  }
  __syncthreads();
  for (int place = threadIdx.x >> 5; place < parts.held; place += Shape<D>::kThreads / 32) {
    const int r = rank * parts.held + place, tok = it.tok0 + r / p.heads, h = it.head0 + r % p.heads;
    if (!(ctl.odd[place / 32] >> (place % 32) & 1u) || !used(r)) continue;
    const int64_t at = it.q0 + (int64_t)tok;
    const int pos = it.m - (it.n - tok);
    const int see_lo = p.window > 0 ? (int)max(INT64_C(0), min((int64_t)it.m, (int64_t)pos - p.window + 1)) : 0;
    const int see_hi = p.causal ? max(0, min(it.m, pos + 1)) : it.m;
    row_again<D>(p, p.q + at * p.q_stride + (int64_t)h * D, p.k + (int64_t)it.k0 * p.k_stride + (int64_t)it.kv * D,
                 p.v + (int64_t)it.k0 * p.v_stride + (int64_t)it.kv * D, see_lo, see_hi, pos,
                 p.slopes != nullptr ? __ldg(p.slopes + h) : 0.f, p.out + at * p.out_stride + (int64_t)h * D,
                 p.lse == nullptr ? nullptr : p.lse + at * p.n_heads + h);
  }
}

// What scores need beyond a scale: nothing, slopes, a cap (and slopes), a cap above kUsualCap
// (and slopes).  Split: a cluster has one item.  (As branches at run time
// these cost the loops registers: 4 x 1000 capped queries of 256 elements 141 us, 157 with
// the caps' two ways, 168 with the split before that; 60 prompts of up to 700
// with slopes 115, so 100.)
enum Options { kNone, kSloped, kCapped, kFar };
template <int D, Options Kind, bool Split, int Terms>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1) prefill_kernel(const __grid_constant__ CUtensorMap tq,
                                                             const __grid_constant__ CUtensorMap tk,
                                                             const __grid_constant__ CUtensorMap tv, const PrefillArgs p) {
  using Z = Shape<D>;
  constexpr int kTiles = Z::kTiles, kKeys = Z::kKeys, kSlots = Z::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];  // query tiles, key and value slots, stages, control
  uint8_t *ring = smem + kTiles * Z::kQTile;
  using Ctl = Control<D>;
  uint8_t *stages = ring + kSlots * Z::kSlot;
  Ctl &ctl = *reinterpret_cast<Ctl *>(stages + 4 * kTiles * kStage);
  auto &q_full = ctl.q_full, &q_empty = ctl.q_empty;
  auto &kv_full = ctl.kv_full, &kv_empty = ctl.kv_empty;
  auto &s_full = ctl.s_full, &p_full = ctl.p_full, &o_full = ctl.o_full;
  auto &item_full = ctl.item_full, &item_empty = ctl.item_empty;
  volatile int &stop = ctl.stop;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < kTiles; ++t) mbar_init(&q_full[t], 1), mbar_init(&q_empty[t], 1);
    for (int s = 0; s < kSlots; ++s) mbar_init(&kv_full[s], 1), mbar_init(&kv_empty[s], 1);
    for (int b = 0; b < 2; ++b) mbar_init(&s_full[b], 1), mbar_init(&p_full[b], 4), mbar_init(&o_full[b], 1);
    for (int b = 0; b < kAhead; ++b) mbar_init(&item_full[b], 1), mbar_init(&item_empty[b], 2 + 4 * kTiles);
    mbar_init(&ctl.answered, 1);
    stop = 0;
    if (Split)
      for (int i = 0; i < 4; ++i) ctl.odd[i] = 0;
    fence_mbar_init();
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  pdl_wait();
  pdl_trigger();
  const int rank = Split ? (int)cluster_rank() : 0;
  bool met = false;  // this warp has been at the cluster's first barrier

  // The items, which warp 2 writes one after another: the other roles take each once.
  int turn = 0;
  uint32_t turn_phase = 0;
  const auto item_ready = [&] {  // false: it gave up
    if (mbar_wait(&item_full[turn], turn_phase, nullptr, p.wait_ns)) return true;
    give_up(&stop, p.err);
    return false;
  };
  if (warp == 0) {
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 0, q_phase = 0;  // q_phase: a bit per tile
      const auto load = [&](const CUtensorMap *map, const Item &it, int j) {
        if (!mbar_wait(&kv_empty[slot], phase ^ 1u, &stop, p.wait_ns)) {
          give_up(&stop, p.err);
          return false;
        }
        mbar_arrive_expect_tx(&kv_full[slot], Z::kSlot);
#pragma unroll
        for (int c = 0; c < Z::kChunks; ++c)
          tma_load_3d(ring + (size_t)slot * Z::kSlot + c * (kKeys * 128), map, 64 * c, it.kv, it.k0 + (it.block0 + (p.slopes == nullptr ? j : -j)) * kKeys, &kv_full[slot]);
        if (++slot == kSlots) slot = 0, phase ^= 1u;
        return true;
      };
      bool ok = true;
      while (ok && item_ready()) {
        const Item &it = ctl.items[turn];
        if (it.n == 0) break;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (it.lo[t] >= it.hi[t]) continue;
          if (!mbar_wait(&q_empty[t], (q_phase >> t & 1u) ^ 1u, &stop, p.wait_ns)) {
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
        if (it.first < it.last) ok = ok && load(&tk, it, it.first);
        if (kTiles == 1 && it.first + 1 < it.last) ok = ok && load(&tk, it, it.first + 1);
        for (int j = it.first; ok && j < it.last; ++j) {
          ok = load(&tv, it, j);
          const int ahead = j + (kTiles == 1 ? 2 : 1);
          if (ok && ahead < it.last) ok = load(&tk, it, ahead);
        }
        if (!ok) break;
        mbar_arrive(&item_empty[turn]);
        if (++turn == kAhead) turn = 0, turn_phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    // The whole warp goes through this in step, one lane issues (see mma_bf16_ss).
    constexpr uint32_t i_s = idesc_bf16(128, kKeys, false), i_o = idesc_bf16(128, D, true);
    const uint32_t leader = elect_lane();
    int slot = 0, step = 0;  // step: of one tile's S buffers
    uint32_t phase = 0, q_phase = 0, p_phase = 0;
    bool ok = true;
    const auto wait = [&](uint64_t *bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, &stop, p.wait_ns));
      if (!ok) give_up(&stop, p.err);
      tc_fence_after();
      return ok;
    };
    // Descriptors differ from the first tile's and slot's in their start address
    // (16-byte units) alone.
    const uint64_t q_desc = sw128_kmajor_desc(smem_u32(smem)), k_desc = sw128_kmajor_desc(smem_u32(ring)),
                   v_desc = sw128_rows_k_desc(smem_u32(ring), kKeys * 128);
    const auto scores = [&](int t, int buf, int s) {  // S[buf] = Q[t] K[slot s]^T
      const uint64_t a = q_desc + (uint64_t)(t * (Z::kQTile / 16)), b = k_desc + (uint64_t)(s * (Z::kSlot / 16));
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_bf16_ss(leader, tmem + Z::kS + buf * kKeys, a + ((k >> 2) * (128 * 128) + (k & 3) * 32) / 16,
                    b + ((k >> 2) * (kKeys * 128) + (k & 3) * 32) / 16, i_s, k > 0 ? 1u : 0u);
      mma_commit_by(leader, &s_full[buf]);
    };
    const auto values = [&](int t, int buf, int s, bool more) {  // O[t] (+)= P[buf] V[slot s]
      const uint64_t b = v_desc + (uint64_t)(s * (Z::kSlot / 16));
#pragma unroll
      for (int k = 0; k < kKeys / 16; ++k) {
        // with two terms the weights of 32 keys lie as 16 columns of the first and 16 of the second
        const uint32_t p0 = tmem + Z::kS + buf * kKeys + (Terms == 1 ? k * 8 : (k >> 1) * 32 + (k & 1) * 8);
        mma_bf16_ts(leader, tmem + Z::kO + t * D, p0, b + k * (2048 / 16), i_o, more || k > 0 ? 1u : 0u);
        if (Terms == 2) mma_bf16_ts(leader, tmem + Z::kO + t * D, p0 + 16, b + k * (2048 / 16), i_o, 1u);
      }
      mma_commit_by(leader, &o_full[buf]);
    };
    const auto release = [&](int s) { mma_commit_by(leader, &kv_empty[s]); };
    const auto next_slot = [&] {
      const int s = slot;
      if (++slot == kSlots) slot = 0, phase ^= 1u;
      return s;
    };
    while (true) {
      if (!(ok = __all_sync(0xffffffffu, item_ready()))) break;
      const Item &it = ctl.items[turn];
      if (uniform(it.n) == 0) break;
      const int first = uniform(it.first), last = uniform(it.last);
      if (first == last) {
      } else if constexpr (kTiles == 2) {
        const int lo[2] = {uniform(it.lo[0]), uniform(it.lo[1])}, hi[2] = {uniform(it.hi[0]), uniform(it.hi[1])};
        // a block of keys has a slot, which both tiles use; of values likewise
        const auto block_scores = [&](int t, int j, int s) {
          if (j == lo[t]) {
            if (!wait(&q_full[t], q_phase >> t & 1u)) return false;
            q_phase ^= 1u << t;
          }
          scores(t, t, s);
          if (hi[t] == j + 1) mma_commit_by(leader, &q_empty[t]);
          return true;
        };
        if (!wait(&kv_full[slot], phase)) break;
        int k_slot = next_slot();
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (ok && lo[t] < hi[t] && lo[t] == first) block_scores(t, first, k_slot);
        if (!ok) break;
        release(k_slot);
        for (int j = first; j < last; ++j) {
          if (!wait(&kv_full[slot], phase)) break;
          const int v_slot = next_slot();
          if (j + 1 < last) {
            if (!wait(&kv_full[slot], phase)) break;
            k_slot = next_slot();
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && lo[t] <= j && j < hi[t]) {
              if (wait(&p_full[t], p_phase >> t & 1u)) values(t, t, v_slot, j > lo[t]);
              p_phase ^= 1u << t;
            }
            if (ok && lo[t] <= j + 1 && j + 1 < hi[t]) block_scores(t, j + 1, k_slot);
          }
          if (!ok) break;
          release(v_slot);
          if (j + 1 < last) release(k_slot);
        }
        if (!ok) break;
      } else {
        if (!wait(&q_full[0], q_phase)) break;
        q_phase ^= 1u;
        const auto block_scores = [&](int j, int buf) {
          if (!wait(&kv_full[slot], phase)) return false;
          const int s = next_slot();
          scores(0, buf, s);
          if (j + 1 == last) mma_commit_by(leader, &q_empty[0]);
          release(s);
          return true;
        };
        for (int j = first; ok && j < last && j < first + 2; ++j) block_scores(j, (step + j - first) & 1);
        for (int j = first; ok && j < last; ++j, ++step) {
          const int buf = step & 1;
          if (!wait(&kv_full[slot], phase) || !wait(&p_full[buf], p_phase >> buf & 1u)) break;
          p_phase ^= 1u << buf;
          const int s = next_slot();
          values(0, buf, s, j > first);
          release(s);
          if (j + 2 < last) block_scores(j + 2, buf);
        }
        if (!ok) break;
      }
      if (lane == 0) mbar_arrive(&item_empty[turn]);
      if (++turn == kAhead) turn = 0, turn_phase ^= 1u;
    }
  } else if (warp == 2) {
    const int groups = p.n_kv * p.chunks, T = item_tokens<D>(p);
    int counts[kHeld];
    const bool held = p.B <= 32 * kHeld;
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int b = 32 * u + lane;
      counts[u] = held && b < p.B ? max(0, clamp_start(p.q_starts, b + 1, p.Tq) - clamp_start(p.q_starts, b, p.Tq) + T - 1) / T : 0;
    }
    int64_t i = Split ? blockIdx.x / p.splits : blockIdx.x;
    uint32_t answer_phase = 0;
    bool ok = true, first = true;
    while (ok) {
      // An item is asked for once there is room to keep it: those that are kept for
      // longer could be another block's.
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&item_empty[turn], turn_phase ^ 1u, &stop, p.wait_ns)))) break;
      Item &it = ctl.items[turn];
      bool some = false;
      while (ok && !some) {
        if (!first) {
          if (Split) {
            i = -1;
          } else if (p.stride > 0) {
            i = i + p.stride < p.items ? i + p.stride : -1;
          } else {
            if (lane == 0) {
              mbar_arrive_expect_tx(&ctl.answered, 16);
              request_block(ctl.answer, &ctl.answered);
            }
            __syncwarp();
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.answered, answer_phase, &stop, p.wait_ns)))) break;
            answer_phase ^= 1u;
            i = requested_block(ctl.answer);
            __syncwarp();
            if (lane == 0) fence_proxy_async_shared();  // the answer has been read before the next is written
          }
        }
        first = false;
        if (i < 0) break;
        const int r = (int)(i / groups), group = (int)(i % groups);
        const Piece at = held ? piece_of(counts, r) : piece_at(p, (int)(p.items / groups) - 1 - r, T);
        some = at.b >= 0 && __shfl_sync(0xffffffffu, lane == 0 && item_of<D, Split>(p, at.b, at.index, group, rank, &it), 0);
      }
      if (!ok) break;
      if (lane == 0) {
        if (!some) it.n = 0;
        mbar_arrive(&item_full[turn]);
      }
      __syncwarp();
      if (!some) break;
      if (++turn == kAhead) turn = 0, turn_phase ^= 1u;
    }
    if (!ok) give_up(&stop, p.err);
  } else if (warp >= 4) {
    // The starts are as they should be: each block that runs looks at all of them, while its
    // first scores are on their way, as which blocks run is not known (another may take over
    // any that has not started).
    bool bad = false;
    for (int b = threadIdx.x - 128; b <= p.B; b += Z::kThreads - 128) {
      const int qs = __ldg(p.q_starts + b), ks = __ldg(p.k_starts + b);
      bad |= qs < 0 || qs > p.Tq || ks < 0 || ks > p.Tk;
      if (b < p.B) bad |= __ldg(p.q_starts + b + 1) < qs || __ldg(p.k_starts + b + 1) < ks;
    }
    if (bad) set_error(p.err, DEV_ERR_BOUNDS);
    __syncwarp();
    constexpr int kParts = kKeys / 32;
    const int t = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int row = (warp & 3) * 32 + lane;  // of the tile
    const uint32_t t_o = tmem + lanes + Z::kO + t * D;
    const int r_tok = row / p.heads, r_head = row - r_tok * p.heads;
    constexpr bool Option = Kind != kNone, usual = Kind != kFar;
    constexpr bool capped = Kind >= kCapped;
    const bool sloped = Kind == kSloped || (capped && p.slopes != nullptr);
    const float unit = capped ? (usual ? 2.f * kLog2e : 1.f) * (p.scale / p.softcap) : 0.f;
    const float scale2 = (!capped ? p.scale : usual ? -2.f * p.softcap : p.softcap) * kLog2e, offset = capped && usual ? p.softcap * kLog2e : 0.f;
    uint32_t step = 0;  // blocks that the tile has had
    // A lane that gives up goes on with the others, over whatever there is, to where the
    // warp votes on it, behind the item's blocks (a warp that was split would not get through
    // its collective instructions, and a vote for each block cost 2% of short prompts).
    const auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (!mbar_wait(bar, parity, &stop, p.wait_ns) && !stop) give_up(&stop, p.err);
      tc_fence_after();
    };
    // The tile's products with V so far.  A barrier per S buffer: when a block's scores
    // are ready the products of the block before it in the same buffer are done, but
    // with one tile not yet those of the other buffer's, and a wait tells only the last
    // of a barrier's phases from the one before it.
    const auto products_done = [&] {
      const uint32_t n = step - 1u;
      kTiles == 2 ? wait(&o_full[t], n & 1u) : wait(&o_full[n & 1u], n >> 1 & 1u);
    };
    while (__all_sync(0xffffffffu, item_ready())) {
      const Item &shared = ctl.items[turn];
      const struct {
        int q0, k0, n, m, tok0, kv, head0, heads;
      } it = {shared.q0, shared.k0, shared.n, shared.m, shared.tok0, shared.kv, shared.head0, shared.heads};
      if (it.n == 0) break;
      // The row's token, of the sequence (past its end: a row of no use); its position is
      // below the last key's by the tokens that follow it.
      const uint32_t tok = (uint32_t)(it.tok0 + t * p.tokens) + (uint32_t)r_tok;
      const bool mine = r_tok < p.tokens && r_head < it.heads && tok < (uint32_t)it.n;
      const int pos = it.m - (int)((uint32_t)it.n - tok);
      // the keys that the row sees
      const int see_lo = p.window > 0 ? (int)max(INT64_C(0), min((int64_t)it.m, (int64_t)pos - p.window + 1)) : 0;
      const int see_hi = p.causal ? max(0, min(it.m, pos + 1)) : it.m;
      const int lo = shared.lo[t], hi = shared.hi[t], whole_lo = shared.whole_lo[t], whole_hi = shared.whole_hi[t];
      const float slope = sloped && mine ? __ldg(p.slopes + it.head0 + r_head) : 0.f, near = slope * kLog2e;
      const uint64_t n01 = pack_f32x2(0.f, near), n23 = pack_f32x2(2.f * near, 3.f * near), n45 = pack_f32x2(4.f * near, 5.f * near),
                     n67 = pack_f32x2(6.f * near, 7.f * near);
      // What a negative slope adds from one block to the one before.  The reference counts
      // on it, up to 2^96 (it may then be that much above the scores); where more than
      // 2^96 would come on top, blocks are read twice.
      const float rise = Option ? fmaxf(-near, 0.f) * kKeys : 0.f;
      const bool steep = Option && __any_sync(0xffffffffu, rise > 192.f);
      const bool rows = __any_sync(0xffffffffu, mine);  // of use in this warp
      float ref = mine ? -INFINITY : 0.f;
      float most = -INFINITY;  // of the blocks so far
      uint64_t sum2[2] = {0, 0};
      float rounding = 0.f;  // of the heaviest weights of the blocks so far
      const int key_step = sloped ? -kKeys : kKeys;
      int key0 = shared.block0 * kKeys + (lo - 1) * key_step;  // the block's first
      for (int j = lo; j < hi; ++j) {
        key0 += key_step;
        const int buf = kTiles == 2 ? t : (int)(step & 1u);
        const bool masked = j < whole_lo || j >= whole_hi;
        const uint32_t t_s = tmem + lanes + Z::kS + buf * kKeys;
        wait(&s_full[buf], (kTiles == 2 ? step : step >> 1) & 1u);
        if (!rows) {
          tc_fence_before();  // of the outputs that the warp read where the products now go
          if (lane == 0) mbar_arrive(&p_full[buf]);
          ++step;
          continue;
        }
        uint32_t s[2][32];
        tmem_ld32(t_s, s[0]);
        // 32 scores in units of log2, options applied and hidden ones -infinity, less the
        // reference.  A slope's share is near * (key - pos): of every eighth key by itself,
        // so that it is off by a unit or two of the distance's.
        const auto exponents = [&](uint32_t(&x)[32], int c0, float minus) {
          if (capped) cap_scores<usual>(x, unit), minus += offset;
          const uint64_t mul = pack_f32x2(scale2, scale2);
          if (sloped) {
            const float base = fmaf(near, (float)(key0 + c0 - pos), minus);
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float eighth = fmaf(near, (float)(c & ~7), base);
              const uint64_t add = add_f32x2(pack_f32x2(eighth, eighth), (c & 7) == 0 ? n01 : (c & 7) == 2 ? n23 : (c & 7) == 4 ? n45 : n67);
              const float2 f = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), mul, add));
              x[c] = __float_as_uint(f.x), x[c + 1] = __float_as_uint(f.y);
            }
          } else {
            const uint64_t add = pack_f32x2(minus, minus);
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float2 f = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), mul, add));
              x[c] = __float_as_uint(f.x), x[c + 1] = __float_as_uint(f.y);
            }
          }
          if (masked) {
            // bit c: key c is before the row's first or behind its last
            const int from = min(max(see_lo - key0 - c0, 0), 32), to = min(max(see_hi - key0 - c0, 0), 32);
            const uint32_t hidden = (uint32_t)((UINT64_C(1) << from) - 1) | ~(uint32_t)((UINT64_C(1) << to) - 1);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (hidden >> c & 1u) x[c] = __float_as_uint(-INFINITY);
          }
        };
        const auto largest = [&](const uint32_t(&x)[32], float top) {
          float other = -INFINITY;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            top = max3(top, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
            other = max3(other, __uint_as_float(x[c + 2]), __uint_as_float(x[c + 3]));
          }
          return fmaxf(top, other);
        };
        const bool twice = steep || __any_sync(0xffffffffu, ref == -INFINITY);
        if (twice) {
          // From the last key that one of the rows sees down, as far as each has seen one:
          // the reference need not be the largest score, and with slopes it is there.
          float top = -INFINITY;
          const int last_key = min(max(see_hi - 1 - key0, 0), kKeys - 1);
          int c = steep ? kKeys - 32 : (int)__reduce_max_sync(0xffffffffu, (unsigned)last_key) & ~31;
#pragma unroll 1
          do {
            tmem_wait_ld(s[0]);
            tmem_ld32(t_s + c, s[0]);
            tmem_wait_ld(s[0]);
            exponents(s[0], c, 0.f);
            top = largest(s[0], top);
            c -= 32;
          } while (c >= 0 && (steep || __any_sync(0xffffffffu, top == -INFINITY)));
          tmem_ld32(t_s, s[0]);
          most = top;
        } else if (Option) {
          most += fminf(rise, 96.f);
        }
        const bool move = most > ref + kMove;
        if (__any_sync(0xffffffffu, move)) {
          // in two factors: what a weight of up to 2^127 leaves may have to come down by more
          // than the smallest factor
          const float keep = !move ? 1.f : ref == -INFINITY ? 0.f : exp2_fast(0.5f * (ref - most));
          const uint64_t keep2 = pack_f32x2(keep, keep);
          if (move) ref = most;
          sum2[0] = mul_f32x2(mul_f32x2(sum2[0], keep2), keep2);
          sum2[1] = mul_f32x2(mul_f32x2(sum2[1], keep2), keep2);
          rounding = rounding * keep * keep;
          if (j > lo) {
            // with two tiles, the products with V are done up to the last block's: they
            // came before this block's scores
            if (kTiles == 1) products_done();
            tmem_wait_ld(s[0]);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(t_o + c, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * keep * keep);
              tmem_st32(t_o + c, o);
            }
          }
        }
        const float minus = ref == -INFINITY ? 0.f : -ref;
        // A weight's steps: exponents of 32 scores, then their exp2, between which the
        // 32 before them are added up, so that the special-function unit always has the
        // next ones.
        [[maybe_unused]] uint32_t second[Terms == 2 ? 16 : 1];
        const auto add_up = [&](uint32_t(&x)[32], int c) {
          const float p0 = __uint_as_float(x[c]), p1 = __uint_as_float(x[c + 1]);
          sum2[c / 2 & 1] = add_f32x2(sum2[c / 2 & 1], pack_f32x2(p0, p1));
          if constexpr (Terms == 1) {
            x[c / 2] = bf16x2_of(p0, p1);
          } else {  // the first 8 bits of each, and the rest rounded
            const uint32_t f0 = x[c] & 0xffff0000u, f1 = x[c + 1] & 0xffff0000u;
            const float2 rest = unpack_f32x2(add_f32x2(pack_f32x2(p0, p1), pack_f32x2(-__uint_as_float(f0), -__uint_as_float(f1))));
            second[c / 2] = bf16x2_of(rest.x, rest.y);
            x[c / 2] = __byte_perm(f0, f1, 0x7632);
          }
        };
        const auto store_weights = [&](uint32_t(&x)[32], int part) {
          tmem_st16(t_s + 16 * Terms * part, x);
          if constexpr (Terms == 2) tmem_st16(t_s + 32 * part + 16, second);
        };
        float top = -INFINITY;  // beyond the reference
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          uint32_t(&x)[32] = s[part & 1], (&before)[32] = s[part & 1 ^ 1];
          tmem_wait_ld(x);
          exponents(x, 32 * part, minus);
          top = largest(x, top);
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            x[c] = __float_as_uint(exp2_in_order(__uint_as_float(x[c])));
            x[c + 1] = __float_as_uint(exp2_in_order(__uint_as_float(x[c + 1])));
            if (part > 0) add_up(before, c);
          }
          // (weights lie over scores that have been read)
          if (part > 0) store_weights(before, part - 1);
          if (part + 1 < kParts) tmem_ld32(t_s + 32 * (part + 1), before);
        }
        uint32_t(&x)[32] = s[kParts - 1 & 1];
#pragma unroll
        for (int c = 0; c < 32; c += 2) add_up(x, c);
        store_weights(x, kParts - 1);
        if constexpr (Terms == 1) {
          const float heaviest = exp2_fast(top);
          rounding += __uint_as_float(bf16x2_of(0.f, heaviest)) - heaviest;
        }
        most = top - minus;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
        ++step;
      }
      if (rows && lo < hi) products_done();
      if (__any_sync(0xffffffffu, stop != 0)) break;
      if (rows) {
      const float2 s0 = unpack_f32x2(sum2[0]), s1 = unpack_f32x2(sum2[1]);
      const float sum = (s0.x + s0.y) + (s1.x + s1.y);
      if constexpr (Split) {
        const Parts parts = Parts::of<D>(p, it.n, it.tok0);
        __syncwarp();
        cluster_sync_all();  // nobody's keys, values and queries are needed any more
        met = true;
        const int r = t * p.tokens * p.heads + row, owner = r / parts.held, slot = rank * parts.held + r - owner * parts.held;
        const bool push = row < p.tokens * p.heads && r < parts.rows;
        const uint32_t to_stats = push ? map_to_rank(smem_u32(smem), (uint32_t)owner) : 0u;
        const uint32_t to = push ? map_to_rank(smem_u32(ring), (uint32_t)owner) + (uint32_t)slot * (D * 4) : 0u;
        if (push) st_cluster8(to_stats + 8 * slot, ref, lo < hi ? log2f(sum) : kNoPart);
        const float inv = sum > 0.f || !(sum == sum) ? 1.f / (sum + rounding) : 0.f;
        if (lo < hi) {
          // by way of the warp's stage, as outputs are below: four rows of 128 bytes at a time
          uint32_t at[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) at[i] = __shfl_sync(0xffffffffu, to, 4 * i + (lane >> 3));
          uint8_t *stage = stages + (warp - 4) * kStage;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + c, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * inv);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              *reinterpret_cast<uint4 *>(stage + lane * 128 + (x ^ (lane & 7)) * 16) = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 f = *reinterpret_cast<const float4 *>(stage + (4 * i + (lane >> 3)) * 128 + ((lane & 7) ^ (4 * i + (lane >> 3) & 7)) * 16);
              if (at[i] != 0) st_cluster16(at[i] + 4 * c + 16 * (lane & 7), f.x, f.y, f.z, f.w);
            }
            __syncwarp();
          }
        }
        break;
      }
      const float inv = sum > 0.f || !(sum == sum) ? 1.f / (sum + rounding) : 0.f;
      // A thread's row of outputs is written by eight lanes, 16 bytes each, so that four
      // rows of 128 bytes leave at a time: through the warp's stage, where the 16-byte
      // pieces of a row are exchanged by its number (a row per lane took five times as
      // long, 32 lines per instruction).
      const int64_t out_at = mine ? (it.q0 + (int64_t)tok) * p.out_stride + (int64_t)(it.head0 + r_head) * D : -1;
      int64_t at[8];  // of the rows that this lane writes pieces of
#pragma unroll
      for (int r = 0; r < 8; ++r) at[r] = __shfl_sync(0xffffffffu, out_at, 4 * r + (lane >> 3));
      const uint64_t inv2 = pack_f32x2(inv, inv);
      uint64_t odd2 = 0;  // outputs times zero: NaN where one is not finite
      uint8_t *stage = stages + (warp - 4) * kStage;
#pragma unroll 1
      for (int c = 0; c < D; c += 64) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t o[32];
          if (lo < hi) {
            tmem_ld32(t_o + c + 32 * h, o);
            tmem_wait_ld(o);
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0;
          }
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const uint64_t two = mul_f32x2(pack_f32x2(__uint_as_float(o[x]), __uint_as_float(o[x + 1])), inv2);
            odd2 = fma_f32x2(two, 0, odd2);
            const float2 f = unpack_f32x2(two);
            o[x / 2] = bf16x2_of(f.x, f.y);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((4 * h + x) ^ (lane & 7)) * 16) =
                make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const uint4 v = *reinterpret_cast<const uint4 *>(stage + (4 * r + (lane >> 3)) * 128 + ((lane & 7) ^ (4 * r + (lane >> 3) & 7)) * 16);
          if (at[r] >= 0) *reinterpret_cast<uint4 *>(p.out + at[r] + c + 8 * (lane & 7)) = v;
        }
        __syncwarp();
      }
      if (mine && p.lse != nullptr)
        p.lse[(it.q0 + (int64_t)tok) * p.n_heads + it.head0 + r_head] = inv == 0.f ? -INFINITY : kLn2 * (ref + log2f(sum));
      __syncwarp();
      const float2 odd = unpack_f32x2(odd2);
      for (uint32_t left = __ballot_sync(0xffffffffu, mine && !(odd.x == 0.f && odd.y == 0.f && sum <= 3.402823466e38f)); left != 0; left &= left - 1) {
        const int from = __ffs(left) - 1;
        const int64_t r = it.q0 + (int64_t)__shfl_sync(0xffffffffu, tok, from);
        const int r_pos = __shfl_sync(0xffffffffu, pos, from), head = it.head0 + __shfl_sync(0xffffffffu, r_head, from);
        const int l = __shfl_sync(0xffffffffu, see_lo, from), h = __shfl_sync(0xffffffffu, see_hi, from);
        row_again<D>(p, p.q + r * p.q_stride + (int64_t)head * D, p.k + (int64_t)it.k0 * p.k_stride + (int64_t)it.kv * D,
                     p.v + (int64_t)it.k0 * p.v_stride + (int64_t)it.kv * D, l, h, r_pos, __shfl_sync(0xffffffffu, slope, from),
                     p.out + r * p.out_stride + (int64_t)head * D, p.lse == nullptr ? nullptr : p.lse + r * p.n_heads + head);
      }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[turn]);
      if (++turn == kAhead) turn = 0, turn_phase ^= 1u;
    }
  }
  if constexpr (Split) {
    // the barriers are met by every warp, whether it gave up or not
    __syncwarp();
    if (!met) cluster_sync_all();
    cluster_sync_all();  // the parts are there
    if (!stop && ctl.items[0].n > 0) join_parts<D>(p, ctl, smem, ring, rank);
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

template <int D, int Terms>
cudaError_t launch_d(PrefillArgs a, int sms, cudaStream_t s) {
  using Z = Shape<D>;
  CUtensorMap tq, tk, tv;
  // without keys nothing of k and v is read
  const bool keys = a.Tk > 0;
  if (!map_rows(&tq, a.q, D, a.n_heads, a.Tq, a.q_stride, a.heads, a.tokens) ||
      !map_rows(&tk, keys ? a.k : a.q, D, keys ? a.n_kv : 1, keys ? a.Tk : 1, keys ? a.k_stride : a.q_stride, 1, Z::kKeys) ||
      !map_rows(&tv, keys ? a.v : a.q, D, keys ? a.n_kv : 1, keys ? a.Tk : 1, keys ? a.v_stride : a.q_stride, 1, Z::kKeys))
    return cudaErrorInvalidValue;
  // a limit on the SMs: so many blocks, and every so-manieth item for each
  a.wait_ns = kWaitNs + kWaitNsPerKey * (uint64_t)a.Tk;
  a.stride = a.splits == 1 && sms > 0 && sms < a.items ? sms : 0;
  const Options kind = a.softcap > kUsualCap ? kFar : a.softcap > 0.f ? kCapped : a.slopes != nullptr ? kSloped : kNone;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.stride > 0 ? a.stride : a.items * a.splits));
  cfg.blockDim = dim3(Z::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D>();
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  const auto whole = kind == kNone ? prefill_kernel<D, kNone, false, Terms>
                     : kind == kSloped ? prefill_kernel<D, kSloped, false, Terms>
                     : kind == kCapped ? prefill_kernel<D, kCapped, false, Terms>
                                       : prefill_kernel<D, kFar, false, Terms>;
  const auto split = kind == kNone ? prefill_kernel<D, kNone, true, Terms>
                     : kind == kSloped ? prefill_kernel<D, kSloped, true, Terms>
                     : kind == kCapped ? prefill_kernel<D, kCapped, true, Terms>
                                       : prefill_kernel<D, kFar, true, Terms>;
  return cudaLaunchKernelEx(&cfg, a.splits > 1 ? split : whole, tq, tk, tv, a);
}

template <int D, int Terms>
cudaError_t ready_d(PrefillFit *fit) {
  for (auto k : {prefill_kernel<D, kNone, false, Terms>, prefill_kernel<D, kSloped, false, Terms>, prefill_kernel<D, kCapped, false, Terms>, prefill_kernel<D, kFar, false, Terms>,
                 prefill_kernel<D, kNone, true, Terms>, prefill_kernel<D, kSloped, true, Terms>, prefill_kernel<D, kCapped, true, Terms>, prefill_kernel<D, kFar, true, Terms>}) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<D>());
    if (e != cudaSuccess) return e;
  }
  for (auto k : {prefill_kernel<D, kNone, true, Terms>, prefill_kernel<D, kSloped, true, Terms>, prefill_kernel<D, kCapped, true, Terms>, prefill_kernel<D, kFar, true, Terms>}) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  // (one CTA fills an SM's shared memory, so the answer is the same for each kernel)
  for (int i = 0; i < kSplitSizes; ++i) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u << i);
    cfg.blockDim = dim3(Shape<D>::kThreads);
    cfg.dynamicSmemBytes = smem_bytes<D>();
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2u << i;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&fit->clusters[i], prefill_kernel<D, kNone, true, Terms>, &cfg);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int Terms>
cudaError_t ready_terms(int d, PrefillFit *fit) {
  return d == 64 ? ready_d<64, Terms>(fit) : d == 128 ? ready_d<128, Terms>(fit) : ready_d<256, Terms>(fit);
}
template <int Terms>
cudaError_t launch_terms(const PrefillArgs &a, int d, int sms, cudaStream_t s) {
  return d == 64 ? launch_d<64, Terms>(a, sms, s) : d == 128 ? launch_d<128, Terms>(a, sms, s) : launch_d<256, Terms>(a, sms, s);
}

}  // namespace
}  // namespace fp8moe
