// Attention of one new token per sequence over a paged key/value cache
// (moe_attn_decode).
//
// out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), in one pass over the keys
// with a running maximum m and sum l per head; when m grows, what was summed
// so far is scaled by e^(m_old - m_new).  Exponentials are taken in base 2,
// the factor log2(e) is part of the scores.
//
// The launch reads each visible key and value row once and is bound by HBM;
// the design keeps loads in flight and everything else out of their way.
//
// Split.  A sequence's visible positions are cut into tiles, a segment is the
// tiles of one (sequence, group of up to 16 query heads that share a key/value
// head), and the list of all segments' tiles is cut evenly over the CTAs,
// whatever the lengths: every CTA finds its piece from the lengths themselves.
// In longer lists a segment counts one tile more, about what its start and end
// cost, or the CTAs that got many short segments would be the last to finish
// (64 sequences of up to 8192: 73 to 100 us at a median of 81 without it).
// A CTA that holds a whole segment writes its result; the parts of a segment
// that several CTAs share go to the workspace as (m, l, unnormalised output)
// and the CTA whose part came last joins them when it is done with its own
// piece, in groups of 16 parts, then the groups.  The order of a join's sums is
// fixed by the parts' places, so results do not depend on the order of arrival.
// No CTA waits for another.
//
// Tile.  Each warp takes 16 or 32 of a tile's keys through its own ring of
// cp.async stages and keeps its own (m, l, output), so the loop
// has no CTA-wide barrier.  S^T = K Q^T and O^T = V^T P^T run as mma.sync
// m16n8k16: 16 keys, then 16 output columns, against 8 query heads (twice for
// groups of 9 to 16), so that few heads leave few lanes idle.  The order of
// the contraction over d and of the output columns is free, so both operands
// are read from shared memory as whole 16-byte pieces of a row: the order
// inside an instruction follows the lanes' pieces, not the row.  Weights pass
// from the scores' layout to the second product's by 8x8 transposes in
// registers (movmatrix).
//
// Maximum.  The reference m of the exponentials is only moved when a score
// exceeds it by 2^8: until then weights are at most 2^8 and every sum is as
// exact as with the true maximum.  Most tiles then cost one vote instead of
// the shuffles and the scaling of the output.
//
// Precision of the weights.
//   bf16 rows: weights need more than bf16's 8 bits, so they are split into a
//   high and a low bf16 part (16 bits together) with a product each.
//   e4m3 rows: codes become f16 (exact), q becomes f16 with a power-of-two
//   shift per head that puts its largest value at 2^14 (exact down to 2^-28 of
//   it), a key's scale multiplies its score, and a value's scale joins the
//   exponent: weights e^(s_j - m') vs_j with a second reference m' for
//   s_j + log2(vs_j), so that they fit f16 whatever the scales.  They are
//   rounded once to f16's 11 bits, an eighth of the step of the bf16 output.
#include "common.cuh"
#include "paged_attn.h"

namespace fp8moe {

namespace {

constexpr int kJoin = 16;              // pieces joined by one CTA
constexpr int kBatch = 8;              // pieces whose loads are in flight together
constexpr int kWeighFrom = 4;          // tiles per CTA from which on a segment counts one more
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLag = 8.f;            // log2 of the largest weight, before its scale
constexpr float kWeightBits = 7.f;     // e4m3: weights are scaled by 2^7, to 2^15 at most

// MH: query heads of a group at most; KM: 16-key steps of a warp's tile; NS:
// stages of a warp's ring; CTAS: that fit on an SM.
constexpr int kSharedBytes = 32;

template <int D_, bool E4M3_, int MH_, int KM_, int kWarps_, int NS_, int CTAS_>
struct Shape {
  static constexpr int D = D_, MH = MH_, KM = KM_, NS = NS_, CTAS = CTAS_;
  static constexpr int kWarps = kWarps_, kThreads = 32 * kWarps;
  static constexpr int kKeys = 16 * KM, kTile = kWarps * kKeys;  // keys of a warp's and a CTA's tile
  static constexpr bool E4M3 = E4M3_;
  static constexpr int NT = MH / 8;                           // columns of 8 heads
  static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
  static constexpr int kPieces = kRowBytes / 16;              // 16-byte pieces of a row
  static constexpr int kHalfTile = kKeys * kRowBytes;         // a warp's K or V rows
  static constexpr int kStage = 2 * kHalfTile + (E4M3 ? 8 * kKeys : 0);
  static constexpr int kRing = kWarps * NS * kStage;
  // values per lane and value row: a 16-byte piece, 8 bytes for the shortest row
  static constexpr int EV = E4M3 && D > 64 ? 16 : 8;
  static constexpr int H = D / (8 * EV);
  static constexpr int kMergeRow = D + 4;                     // floats; the odd pieces spread banks
  static constexpr int kMerge = kWarps * MH * kMergeRow * 4;  // f32 outputs of the warps
  static constexpr int kSmem = kRing + kMerge + kWarps * MH * 8 + MH * D * 2 + 2 * kSharedBytes;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// 16 / 4 bytes to shared memory, zeros where !on.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Four e4m3 codes as two f16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t &lo, uint32_t &hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// Transpose of an 8x8 matrix of 16-bit values held two per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float lds4(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^x to two units in the last place of f32, 0 below 2^-126.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^(from - to), the factor of a state whose maximum was `from` under the
// maximum `to` >= from.  A state with no maximum yet holds zeros, or NaN,
// which any factor keeps.
__device__ __forceinline__ float rescale(float from, float to) {
  return from == -INFINITY ? 1.f : ex2(from - to);
}

// tanh: an odd polynomial below 0.6 (least-squares fit of the relative error
// over Chebyshev points, 3e-9), (1 - t) / (1 + t) with t = e^(-2|y|) above.
__device__ __forceinline__ float tanh_f32(float y) {
  const float z = y * y;
  float p = fmaf(z, -0.005895158741623163f, 0.020795973017811775f);
  p = fmaf(z, p, -0.053783830255270004f);
  p = fmaf(z, p, 0.13331924378871918f);
  p = fmaf(z, p, -0.33333298563957214f);
  const float small = fmaf(y * z, p, y);
  const float t = ex2(-2.f * kLog2e * fabsf(y));
  const float large = copysignf(__fdividef(1.f - t, 1.f + t), y);
  return fabsf(y) < 0.6f ? small : large;
}

// Two weights in 16 bits each, and what the bf16 pair leaves of them.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (F16) return pack_f16x2(a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2_rest(float a, float b, uint32_t high) {
  return pack2<false>(a - __uint_as_float(high << 16), b - __uint_as_float(high & 0xffff0000u));
}

// Visible positions of a sequence, and the tiles of T positions they touch.
struct Span {
  int lo, hi;      // [lo, hi); hi is the length
  int first, n;    // first tile, number of tiles (one, all hidden, if none is visible)
};
template <int T>
__device__ __forceinline__ Span span_of(const DecodeArgs &a, int b) {
  int len = a.lens[b];
  if (len < 0) len = 0;
  if (len > a.capacity) len = (int)a.capacity;
  int lo = a.starts ? a.starts[b] : 0;
  if (lo < 0) lo = 0;
  if (a.window > 0 && lo < len - a.window) lo = len - a.window;
  Span s{lo, len, lo / T, 1};
  if (lo < len) s.n = (len + T - 1) / T - s.first;
  return s;
}

// A place in the list of all tiles: tile `tile` of head group `hg` of
// key/value head `ch` of sequence b.
template <int T>
struct Cursor {
  int b, ch, hg, tile;
  Span s;
  __device__ __forceinline__ void next(const DecodeArgs &a) {
    if (++tile < s.n) return;
    tile = 0;
    if (++hg < a.groups_per_kv) return;
    hg = 0;
    if (++ch < a.n_kv) return;
    ch = 0;
    if (++b < a.B) s = span_of<T>(a, b);
  }
};

// The even cut of W units over N CTAs: the first W % N take one more.
struct Cut {
  uint32_t each, more;
  __device__ __forceinline__ Cut(uint32_t W, uint32_t N) : each(W / N), more(W % N) {}
  __device__ __forceinline__ uint32_t start(uint32_t cta) const { return each * cta + min(cta, more); }
  __device__ __forceinline__ uint32_t owner(uint32_t unit) const {
    const uint32_t big = more * (each + 1);
    return unit < big ? unit / (each + 1) : more + (unit - big) / each;
  }
};

// A segment that other CTAs hold parts of, written to the workspace: it is
// joined when this CTA is done, if its part was the last to arrive.
struct Shared {
  int b, ch, hg;
  uint32_t first, parts, last;  // CTA of the first part, number of parts, whether to join
  uint32_t unused[2];
};

template <class S>
__global__ void __launch_bounds__(S::kThreads, S::CTAS) decode_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int D = S::D, MH = S::MH, NT = S::NT, NS = S::NS, EV = S::EV, KM = S::KM;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kKeys = S::kKeys, kTile = S::kTile;
  constexpr bool Q8 = S::E4M3;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;  // row and column of the matrix instructions
  float *merge = reinterpret_cast<float *>(smem + S::kRing);            // [warp][MH][kMergeRow]
  float2 *ml = reinterpret_cast<float2 *>(smem + S::kRing + S::kMerge);  // [warp][MH]
  uint4 *qbuf = reinterpret_cast<uint4 *>(smem + S::kRing + S::kMerge + kWarps * MH * 8);  // [MH][D / 8]
  Shared *shared = reinterpret_cast<Shared *>(qbuf + MH * D / 8);                         // [2]
  static_assert(sizeof(Shared) == kSharedBytes, "two of them fit");

  // ---- this CTA's piece [t0, t1) of the W tiles of all sequences
  const auto count = [&](int b, Span *sp) {
    const int len = a.lens[b];
    if (len < 0 || len > a.capacity) set_error(a.err, DEV_ERR_BOUNDS);
    *sp = span_of<kTile>(a, b);
    return (uint32_t)(sp->n * a.n_groups);
  };
  const auto scan = [&](uint32_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    return v;
  };
  // The place of a unit: the tile it is or comes before, and the cursor there.
  // `before`: tiles of the sequences before k.b, whose span is k.s.
  uint32_t extra = 0;  // units of a segment beyond its tiles
  const auto place = [&](uint32_t unit, uint32_t before, Cursor<kTile> &k) {
    const uint32_t r = unit - before - extra * (uint32_t)(a.n_groups * k.b);
    const int vh = (int)(r / (k.s.n + extra));
    k.tile = (int)r - vh * (int)(k.s.n + extra);
    k.ch = vh / a.groups_per_kv;
    k.hg = vh - k.ch * a.groups_per_kv;
    return before + vh * k.s.n + k.tile;
  };
  uint32_t W, t0, t1, n_ctas;
  Cursor<kTile> cu;
  if (a.B <= 32) {  // a sequence per lane, every warp for itself
    Span sp{0, 0, 0, 0};
    const uint32_t n = lane < a.B ? count(lane, &sp) : 0;
    const uint32_t incl = scan(n);
    W = __shfl_sync(0xffffffffu, incl, 31);
    n_ctas = min(W, gridDim.x);
    if (blockIdx.x >= n_ctas) return;
    extra = W >= kWeighFrom * gridDim.x ? 1 : 0;
    const uint32_t units = W + extra * (uint32_t)(a.n_groups * a.B);
    const Cut cut(units, n_ctas);
    const uint32_t end = incl + extra * (uint32_t)(a.n_groups * (lane + 1));  // in units
    const auto at = [&](uint32_t unit, Cursor<kTile> &k) {
      const int b = __ffs((int)__ballot_sync(0xffffffffu, end > unit && lane < a.B)) - 1;
      k.b = b;
      k.s.lo = __shfl_sync(0xffffffffu, sp.lo, b);
      k.s.hi = __shfl_sync(0xffffffffu, sp.hi, b);
      k.s.first = __shfl_sync(0xffffffffu, sp.first, b);
      k.s.n = __shfl_sync(0xffffffffu, sp.n, b);
      return place(unit, __shfl_sync(0xffffffffu, incl - n, b), k);
    };
    t0 = at(cut.start(blockIdx.x), cu);
    t1 = W;
    if (blockIdx.x + 1 < n_ctas) {
      Cursor<kTile> k;
      t1 = at(cut.start(blockIdx.x + 1), k);
    }
  } else {  // a run of sequences per thread
    uint32_t *sums = reinterpret_cast<uint32_t *>(merge), *found = sums + kWarps;
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
    Span sp;
    uint32_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += count(b, &sp);
    uint32_t incl = scan(mine);
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    W = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += sums[w];
      W += sums[w];
    }
    n_ctas = min(W, gridDim.x);
    if (blockIdx.x >= n_ctas) return;
    extra = W >= kWeighFrom * gridDim.x ? 1 : 0;
    const uint32_t units = W + extra * (uint32_t)(a.n_groups * a.B);
    const Cut cut(units, n_ctas);
    const auto in_units = [&](uint32_t tiles, int b) { return tiles + extra * (uint32_t)(a.n_groups * b); };
    for (int i = 0; i < 2; ++i) {  // the thread whose run holds it finds the first unit, and the next CTA's
      const uint32_t unit = cut.start(blockIdx.x + i);
      if (in_units(incl - mine, b0) <= unit && unit < in_units(incl, b1)) {
        uint32_t at = incl - mine;
        int b = b0;
        for (;; ++b) {
          const uint32_t n = (uint32_t)(span_of<kTile>(a, b).n * a.n_groups);
          if (unit < in_units(at + n, b + 1)) break;
          at += n;
        }
        found[2 * i] = b;
        found[2 * i + 1] = at;
      }
    }
    __syncthreads();
    cu.b = found[0];
    cu.s = span_of<kTile>(a, cu.b);
    t0 = place(cut.start(blockIdx.x), found[1], cu);
    t1 = W;
    if (blockIdx.x + 1 < n_ctas) {
      Cursor<kTile> k;
      k.b = found[2];
      k.s = span_of<kTile>(a, k.b);
      t1 = place(cut.start(blockIdx.x + 1), found[3], k);
    }
    __syncthreads();  // the merge buffer is free again
  }
  if (t0 >= t1) return;  // a piece of nothing but a segment's end
  if (cu.tile == cu.s.n) {  // it begins with one
    --cu.tile;
    cu.next(a);
  }
  const int n_tiles = (int)(t1 - t0);
  const Cut cut(W + extra * (uint32_t)(a.n_groups * a.B), n_ctas);
  const int G = a.n_heads / a.n_kv;

  // ---- loads: the rows of a warp's keys, NS stages ahead of their use
  constexpr int kRowsAtOnce = 32 / S::kPieces;  // rows of one copy instruction
  constexpr uint32_t kAll = kKeys == 32 ? 0xffffffffu : (1u << kKeys) - 1;
  const uint32_t ring = smem_addr(smem) + warp * (NS * S::kStage);
  const int my_key = lane & (kKeys - 1), my_row = lane / S::kPieces, my_piece = lane % S::kPieces;
  const int64_t my_off = my_row * a.kv.slot_stride + my_piece * 16;
  const int64_t row_step = kRowsAtOnce * a.kv.slot_stride;
  Cursor<kTile> ld = cu;
  int ld_left = n_tiles;
  int32_t page = -1;          // page of this lane's key in the next tile to load
  int64_t row = 0, srow = 0;  // offsets of its row and its scales
  uint32_t on = 0;            // keys of the tile that are loaded
  auto key_of = [&](const Cursor<kTile> &k) { return (k.s.first + k.tile) * kTile + warp * kKeys; };
  auto touches = [&](const Cursor<kTile> &k) {
    const int base = key_of(k);
    return base < k.s.hi && base + kKeys > k.s.lo;
  };
  auto page_index = [&](int j) { return (int)(((uint64_t)(uint32_t)j * a.page_mul) >> a.page_shift); };
  auto fetch_page = [&]() {
    if (ld_left <= 0) return;
    const int j = key_of(ld) + my_key;
    page = -1;
    if (j >= ld.s.lo && j < ld.s.hi) page = a.table[ld.b * a.table_stride + page_index(j)];
  };
  auto load_half = [&](int stage, bool is_v) {
    if (ld_left > 0 && touches(ld)) {
      const uint32_t dst = ring + stage * S::kStage + (is_v ? S::kHalfTile : 0);
      if (!is_v) {  // where the keys lie; the same for their value rows
        const int j = key_of(ld) + my_key;
        const bool good = (uint32_t)page < (uint32_t)a.kv.n_pages;
        if (!good && j >= ld.s.lo && j < ld.s.hi) set_error(a.err, DEV_ERR_BOUNDS);
        on = __ballot_sync(0xffffffffu, good) & kAll;
        const int slot = j - page_index(j) * a.kv.page_size;
        row = good ? page * a.kv.page_stride + ld.ch * a.kv.head_stride + slot * a.kv.slot_stride : 0;
        if (Q8)
          srow = good ? page * a.kv.scale_page_stride + ld.ch * a.kv.scale_head_stride +
                            slot * a.kv.scale_slot_stride
                      : 0;
      }
      const uint8_t *base = is_v ? a.kv.v : a.kv.k;
      // 16-byte pieces are exchanged within a row so that the reads below hit
      // all banks
      const auto place_of = [&](int i) {
        const int r = i * kRowsAtOnce + my_row;
        int q = my_piece;
        if (S::kPieces >= 8) q ^= is_v ? (r & 6) : ((r & 1) << 2);
        else if (is_v) q ^= (r >> 1) & 3;
        return dst + r * S::kRowBytes + q * 16;
      };
      if (a.whole_pages && on == kAll) {  // each 16 keys lie in one page
#pragma unroll
        for (int t = 0; t < KM; ++t) {
          const uint8_t *p = base + __shfl_sync(0xffffffffu, row, 16 * t) + my_off;
#pragma unroll
          for (int i = 0; i < 16 / kRowsAtOnce; ++i) {
            copy16(place_of(t * (16 / kRowsAtOnce) + i), p);
            p += row_step;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kKeys / kRowsAtOnce; ++i) {
          const int r = i * kRowsAtOnce + my_row;
          copy16(place_of(i), base + __shfl_sync(0xffffffffu, row, r) + my_piece * 16, (on >> r) & 1);
        }
      }
      if (Q8 && !is_v) {  // both scales of a key come with its key row
        const uint32_t sdst = ring + stage * S::kStage + 2 * S::kHalfTile + 4 * my_key;
        const bool take = (on >> my_key) & 1;
        if (kKeys == 32 || lane < kKeys) copy4(sdst, a.kv.k_scale + srow, take);
        if (kKeys == 32 || lane >= kKeys) copy4(sdst + 4 * kKeys, a.kv.v_scale + srow, take);
      }
    }
    copy_commit();
    if (is_v && --ld_left > 0) {
      ld.next(a);
      fetch_page();
    }
  };
  fetch_page();
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    load_half(s, false);
    load_half(s, true);
  }

  // ---- the segment's state; heads 8n + 2c and 8n + 2c + 1 are this lane's
  uint32_t qf[NT][D / 16][2];
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2], mv[NT][2];  // mv: the reference of weights with value scales
  float qs[NT][2], sl[NT][2];           // scale of a raw score, slope * log2(e)
  const float cap2 = a.softcap * kLog2e;
  const bool plain = !(a.softcap > 0.f) && a.slopes == nullptr;
  // a segment's queries on their way to shared memory: loaded while the one
  // before it is finished
  constexpr int kQPieces = (MH * D / 8 + kThreads - 1) / kThreads;
  const auto fetch_q = [&](const Cursor<kTile> &k, uint4 (&w)[kQPieces]) {
    const int in_kv = k.hg * a.group, heads = min(a.group, G - in_kv);
    const __nv_bfloat16 *q = a.q + (int64_t)k.b * a.q_stride + (int64_t)(k.ch * G + in_kv) * D;
#pragma unroll
    for (int i = 0; i < kQPieces; ++i) {
      const int p = threadIdx.x + i * kThreads;
      w[i] = p < heads * (D / 8) ? reinterpret_cast<const uint4 *>(q)[p] : make_uint4(0, 0, 0, 0);
    }
  };
  const auto put_q = [&](const uint4 (&w)[kQPieces]) {
#pragma unroll
    for (int i = 0; i < kQPieces; ++i)
      if ((int)threadIdx.x + i * kThreads < MH * (D / 8)) qbuf[threadIdx.x + i * kThreads] = w[i];
  };
  auto start_segment = [&]() {
    const int in_kv = cu.hg * a.group;
    const int heads = min(a.group, G - in_kv), head0 = cu.ch * G + in_kv;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
      const int h = g + 8 * n;  // the head whose q this lane holds
      uint4 w[D / 32];
#pragma unroll
      for (int s = 0; s < D / 32; ++s) {
        // bf16: piece c + 4s of 8 elements; e4m3: halves of piece c + 4 (s / 2) of 16
        const int at = Q8 ? (c + 4 * (s / 2)) * 16 + 8 * (s & 1) : (c + 4 * s) * 8;
        w[s] = qbuf[(h * D + at) / 8];
      }
      float unit = a.scale;
      if (!Q8) {
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
          qf[n][2 * s][0] = w[s].x;
          qf[n][2 * s][1] = w[s].y;
          qf[n][2 * s + 1][0] = w[s].z;
          qf[n][2 * s + 1][1] = w[s].w;
        }
      } else {
        float big = 0.f;
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = u4_word(w[s], i);
            const float x = fabsf(__uint_as_float(v << 16)), y = fabsf(__uint_as_float(v & 0xffff0000u));
            if (x < INFINITY) big = fmaxf(big, x);
            if (y < INFINITY) big = fmaxf(big, y);
          }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        int e = 15;
        if (big > 0.f) frexpf(big, &e);
        const Pow2 up = pow2_factors(15 - e);
        const Pow2 down = pow2_factors(e - 15);
        unit = down(a.scale);
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = u4_word(w[s], i);
            qf[n][2 * s + i / 2][i & 1] =
                pack_f16x2(up(__uint_as_float(v << 16)), up(__uint_as_float(v & 0xffff0000u)));
          }
      }
      unit = a.softcap > 0.f ? unit / a.softcap : unit * kLog2e;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        m[n][u] = mv[n][u] = -INFINITY;
        l[n][u] = 0.f;
        qs[n][u] = __shfl_sync(0xffffffffu, unit, 8 * c + 4 * u);
        const int hh = 8 * n + 2 * c + u;
        sl[n][u] = a.slopes && hh < heads ? a.slopes[head0 + hh] * kLog2e : 0.f;
      }
    }
  };

  // ---- one tile of a warp
  // Raw scores, and the keys' scales (vs: log2): value i of step t is key
  // 16t + g + 8 (i / 2).  After this the stage's key rows and scales are free.
  auto scores = [&](int stage, float (&s)[KM][NT][4], float (&ks)[KM][2], float (&vs)[KM][2]) {
    const uint32_t base = ring + stage * S::kStage;
    if (Q8) {
#pragma unroll
      for (int t = 0; t < KM; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t at = base + 2 * S::kHalfTile + 4 * (16 * t + g + 8 * u);
          ks[t][u] = lds4(at);
          vs[t][u] = lg2(lds4(at + 4 * kKeys));
        }
    }
#pragma unroll
    for (int t = 0; t < KM; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][n][i] = 0.f;
    const int swz = S::kPieces >= 8 ? (g & 1) << 2 : 0;  // the same for all of this lane's rows
    const uint32_t row0 = base + g * S::kRowBytes;
#pragma unroll
    for (int i = 0; i < S::kPieces / 4; ++i) {
      const uint32_t at = row0 + (((c + 4 * i) ^ swz) << 4);
#pragma unroll
      for (int t = 0; t < KM; ++t) {
        const uint4 k0 = lds16(at + 16 * t * S::kRowBytes);
        const uint4 k1 = lds16(at + (16 * t + 8) * S::kRowBytes);
        if (!Q8) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816<false>(s[t][n], k0.x, k1.x, k0.y, k1.y, qf[n][2 * i][0], qf[n][2 * i][1]);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816<false>(s[t][n], k0.z, k1.z, k0.w, k1.w, qf[n][2 * i + 1][0], qf[n][2 * i + 1][1]);
        } else {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16(u4_word(k0, w), a0, a2);
            e4m3x4_to_f16(u4_word(k1, w), a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816<true>(s[t][n], a0, a1, a2, a3, qf[n][4 * i + w][0], qf[n][4 * i + w][1]);
          }
        }
      }
    }
  };
  // Weights of the tile's keys, transposed to (head g; keys 16t + 2c, + 1) and
  // (.., keys 16t + 8 + 2c, + 1): high parts, and what they leave.
  auto weights = [&](float (&s)[KM][NT][4], const float (&ks)[KM][2], const float (&vs)[KM][2],
                     uint32_t (&p_hi)[KM][NT][2], uint32_t (&p_lo)[KM][NT][2]) {
    const int base = key_of(cu);
#pragma unroll
    for (int t = 0; t < KM; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][n][i] *= Q8 ? qs[n][i & 1] * ks[t][i >> 1] : qs[n][i & 1];
    if (!plain) {
#pragma unroll
      for (int t = 0; t < KM; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = s[t][n][i];
            if (a.softcap > 0.f) x = cap2 * tanh_f32(x);
            const int key = base + 16 * t + g + 8 * (i >> 1);
            s[t][n][i] = fmaf(sl[n][i & 1], (float)(key - (cu.s.hi - 1)), x);
          }
    }
    if (base < cu.s.lo || base + kKeys > cu.s.hi) {
#pragma unroll
      for (int t = 0; t < KM; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = base + 16 * t + g + 8 * (i >> 1);
          if (key < cu.s.lo || key >= cu.s.hi) {
#pragma unroll
            for (int n = 0; n < NT; ++n) s[t][n][i] = -INFINITY;
          }
        }
    }
    bool high = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float top = fmaxf(s[0][n][u], s[0][n][2 + u]);
        if (KM == 2) top = fmaxf(top, fmaxf(s[KM - 1][n][u], s[KM - 1][n][2 + u]));
        high |= top > m[n][u] + kLag;
        if (Q8) {
          top = fmaxf(s[0][n][u] + vs[0][0], s[0][n][2 + u] + vs[0][1]);
          if (KM == 2) top = fmaxf(top, fmaxf(s[KM - 1][n][u] + vs[KM - 1][0], s[KM - 1][n][2 + u] + vs[KM - 1][1]));
          high |= top > mv[n][u] + kLag;
        }
      }
    if (__any_sync(0xffffffffu, high)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float top = -INFINITY, top_v = -INFINITY;
#pragma unroll
          for (int t = 0; t < KM; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              top = fmaxf(top, s[t][n][2 * i + u]);
              if (Q8) top_v = fmaxf(top_v, s[t][n][2 * i + u] + vs[t][i]);
            }
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            if (Q8) top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, x));
          }
          top = fmaxf(top, m[n][u]);
          float keep = rescale(m[n][u], top);
          l[n][u] *= keep;
          m[n][u] = top;
          if (Q8) {
            top_v = fmaxf(top_v, mv[n][u]);
            keep = rescale(mv[n][u], top_v);
            mv[n][u] = top_v;
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[n][i][u] *= keep;
            o[n][i][2 + u] *= keep;
          }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float zero[2], zero_v[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        zero[u] = m[n][u] == -INFINITY ? 0.f : m[n][u];
        if (Q8) zero_v[u] = (mv[n][u] == -INFINITY ? 0.f : mv[n][u]) - kWeightBits;
      }
#pragma unroll
      for (int t = 0; t < KM; ++t) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = ex2(s[t][n][i] - zero[i & 1]);
          l[n][i & 1] += p[i];
          if (Q8) p[i] = ex2(s[t][n][i] + (vs[t][i >> 1] - zero_v[i & 1]));
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t hi = pack2<Q8>(p[2 * u], p[2 * u + 1]);
          p_hi[t][n][u] = transpose8(hi);
          if (!Q8) p_lo[t][n][u] = transpose8(pack2_rest(p[2 * u], p[2 * u + 1], hi));
        }
      }
    }
  };
  auto add_values = [&](int stage, const uint32_t (&p_hi)[KM][NT][2], const uint32_t (&p_lo)[KM][NT][2]) {
    const uint32_t vb = ring + stage * S::kStage + S::kHalfTile;
#pragma unroll
    for (int t = 0; t < KM; ++t)
#pragma unroll
      for (int h = 0; h < S::H; ++h) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * c + (i & 1) + 8 * (i >> 1);  // r & 6 is 2c for all four
          const uint32_t row_at = vb + (16 * t + r) * S::kRowBytes;
          if (S::kPieces >= 8) {
            v[i] = lds16(row_at + (((g + 8 * h) ^ (2 * c)) << 4));
          } else {  // rows of 64 bytes, half a piece per lane
            const uint2 x = lds8(row_at + (((g >> 1) ^ c) << 4) + 8 * (g & 1));
            v[i] = make_uint4(x.x, x.y, 0, 0);
          }
        }
#pragma unroll
        for (int w = 0; w < (Q8 ? EV / 4 : 4); ++w) {
          const uint32_t v0 = u4_word(v[0], w), v1 = u4_word(v[1], w), v2 = u4_word(v[2], w),
                         v3 = u4_word(v[3], w);
          if (!Q8) {  // columns 2w, 2w + 1 of the piece, keys paired
            const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
            const uint32_t a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816<false>(o[n][4 * h + w], a0, a1, a2, a3, p_hi[t][n][0], p_hi[t][n][1]);
              mma16816<false>(o[n][4 * h + w], a0, a1, a2, a3, p_lo[t][n][0], p_lo[t][n][1]);
            }
          } else {
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // columns 4w + 2u, + 1
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(__byte_perm(v0, v1, u ? 0x7362 : 0x5140), a0, a1);
              e4m3x4_to_f16(__byte_perm(v2, v3, u ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816<true>(o[n][EV / 2 * h + 2 * w + u], a0, a1, a2, a3, p_hi[t][n][0], p_hi[t][n][1]);
            }
          }
        }
      }
  };

  // ---- end of a segment, or of this CTA's piece of it
  // Outputs are handled as float4 items: item i of a head is elements 4i .. 4i + 3.
  auto write_out = [&](int b, int head, int item, float4 v, float mm, float ll) {
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const int64_t bh = (int64_t)b * a.n_heads + head;
    uint2 w;
    w.x = pack2<false>(v.x * inv, v.y * inv);
    w.y = pack2<false>(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2 *>(a.out + bh * D + 4 * item) = w;
    if (item == 0 && a.lse) a.lse[bh] = (mm + log2f(ll)) * kLn2;
  };
  float4 *part = reinterpret_cast<float4 *>(a.part);
  float2 *part_ml = reinterpret_cast<float2 *>(a.part_ml);
  // a CTA's own slots: 0 for a segment that began before its piece, 1 otherwise
  const auto slot_of = [&](int first, int nth) { return 2 * (first + nth) + (nth == 0 ? 1 : 0); };
  // Thread 0: counts a part that all threads have written; true for the last.
  const auto arrive = [&](int *counter, int n) {
    __threadfence();
    const bool last = atomicAdd(counter, 1) == n - 1;
    if (last) *counter = 0;  // for the next call
    __threadfence();
    return last;
  };
  int n_shared = 0;
  // Ends the segment of tiles [seg0, seg1), or this CTA's part of it; w: the next one's queries.
  auto finish_segment = [&](uint32_t seg0, uint32_t seg1, const uint4 (&w)[kQPieces]) {
    const int in_kv = cu.hg * a.group, heads = min(a.group, G - in_kv);
    const int head0 = cu.ch * G + in_kv;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float sum = l[n][u];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        float f = 1.f;
        if (Q8 && m[n][u] != -INFINITY && mv[n][u] != -INFINITY) f = ex2(mv[n][u] - m[n][u] - kWeightBits);
        const int h = 8 * n + 2 * c + u;
        if (h < heads) {
          float *dst = merge + (warp * MH + h) * S::kMergeRow;
#pragma unroll
          for (int hh = 0; hh < S::H; ++hh)
#pragma unroll
            for (int jj = 0; jj < EV / 4; ++jj) {
              const float *x = o[n][EV / 2 * hh + 2 * jj], *y = o[n][EV / 2 * hh + 2 * jj + 1];
              *reinterpret_cast<float4 *>(dst + (g + 8 * hh) * EV + 4 * jj) =
                  make_float4(x[u] * f, x[2 + u] * f, y[u] * f, y[2 + u] * f);
            }
          if (g == 0) ml[warp * MH + h] = make_float2(m[n][u], sum);
        }
      }
    __syncthreads();
    put_q(w);
    // the CTAs that hold parts of this segment
    int first = blockIdx.x, parts = 1;
    if (seg0 < t0 || seg1 > t1) {
      const uint32_t ends = extra * (uint32_t)(cu.b * a.n_groups + cu.ch * a.groups_per_kv + cu.hg);
      first = (int)cut.owner(seg0 + ends);
      parts = (int)cut.owner(seg1 - 1 + ends) - first + 1;
    }
    const int items = heads * (D / 4);
    const int mine = slot_of(first, blockIdx.x - first);
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const int h = i / (D / 4), it = i % (D / 4);
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[w * MH + h].x);
      float ll = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 s = ml[w * MH + h];
        const float f = rescale(s.x, mm);
        const float4 x = *reinterpret_cast<const float4 *>(merge + (w * MH + h) * S::kMergeRow + 4 * it);
        ll = fmaf(f, s.y, ll);
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
      }
      if (parts == 1) {
        write_out(cu.b, head0 + h, it, v, mm, ll);
      } else {
        part[((int64_t)mine * a.group + h) * (D / 4) + it] = v;
        if (it == 0) part_ml[(int64_t)mine * a.group + h] = make_float2(mm, ll);
      }
    }
    __syncthreads();  // the part is written, and the merge buffer free again
    if (parts > 1) {
      if (threadIdx.x == 0) {
        const int grp = (blockIdx.x - first) / kJoin, p0 = grp * kJoin;
        shared[n_shared] = Shared{cu.b, cu.ch, cu.hg, (uint32_t)first, (uint32_t)parts,
                                  arrive(a.counters + (grp == 0 ? 0 : a.max_ctas) + first + p0,
                                         min(kJoin, parts - p0)), {0, 0}};
      }
      ++n_shared;
    }
  };
  // Joins this CTA's group of the segment's parts, then, if that was the last
  // group, the groups.  Counters: a CTA is the first of at most one shared
  // segment and a later one of at most one other, so three arrays by CTA do.
  auto join_shared = [&](const Shared &sh) {
    const int first = sh.first, parts = sh.parts;
    const int in_kv = sh.hg * a.group, heads = min(a.group, G - in_kv);
    const int head0 = sh.ch * G + in_kv, items = heads * (D / 4);
    auto join = [&](int p0, int step, int n, bool final) {
      for (int i = threadIdx.x; i < items; i += kThreads) {
        const int h = i / (D / 4), it = i % (D / 4);
        float mm = -INFINITY, ll = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < n; p += kBatch) {
          float2 s[kBatch];
          float4 x[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            s[k] = make_float2(-INFINITY, 0.f);
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p + k < n) {
              const int64_t at = (int64_t)slot_of(first, p0 + (p + k) * step) * a.group + h;
              s[k] = __ldcg(part_ml + at);
              x[k] = __ldcg(part + at * (D / 4) + it);
            }
          }
          float top = mm;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) top = fmaxf(top, s[k].x);
          const float f0 = rescale(mm, top);
          ll *= f0;
          v.x *= f0;
          v.y *= f0;
          v.z *= f0;
          v.w *= f0;
          mm = top;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const float f = rescale(s[k].x, top);
            ll = fmaf(f, s[k].y, ll);
            v.x = fmaf(f, x[k].x, v.x);
            v.y = fmaf(f, x[k].y, v.y);
            v.z = fmaf(f, x[k].z, v.z);
            v.w = fmaf(f, x[k].w, v.w);
          }
        }
        if (final) {
          write_out(sh.b, head0 + h, it, v, mm, ll);
        } else {  // in place of the group's first piece, which only this thread has read ..
          part[((int64_t)slot_of(first, p0) * a.group + h) * (D / 4) + it] = v;
          if (it == 0) ml[h] = make_float2(mm, ll);  // .. except for its statistics
        }
      }
      if (!final) {
        __syncthreads();
        for (int h = threadIdx.x; h < heads; h += kThreads)
          part_ml[(int64_t)slot_of(first, p0) * a.group + h] = ml[h];
      }
    };
    const int p0 = ((int)blockIdx.x - first) / kJoin * kJoin, in_grp = min(kJoin, parts - p0);
    const int groups = (parts + kJoin - 1) / kJoin;
    join(p0, 1, in_grp, groups == 1);
    if (groups > 1) {
      __syncthreads();
      if (threadIdx.x == 0) shared[0].last = arrive(a.counters + 2 * a.max_ctas + first, groups);
      __syncthreads();
      if (shared[0].last) join(0, kJoin, groups, true);
    }
  };

  {
    uint4 w[kQPieces];
    fetch_q(cu, w);
    put_q(w);
    __syncthreads();
  }
  start_segment();
  int stage = 0;
  for (int i = 0; i < n_tiles; ++i) {
    const bool busy = touches(cu);
    uint32_t p_hi[KM][NT][2], p_lo[KM][NT][2];
    float s[KM][NT][4], ks[KM][2], vs[KM][2];
    copy_wait<2 * NS - 1>();  // the key rows
    __syncwarp();
    if (busy) scores(stage, s, ks, vs);
    __syncwarp();
    load_half(stage, false);
    if (busy) weights(s, ks, vs, p_hi, p_lo);
    copy_wait<2 * NS - 1>();  // the value rows
    __syncwarp();
    if (busy) add_values(stage, p_hi, p_lo);
    __syncwarp();
    load_half(stage, true);
    const bool last = i == n_tiles - 1;
    if (last || cu.tile == cu.s.n - 1) {
      Cursor<kTile> nx = cu;
      uint4 w[kQPieces] = {};
      if (!last) {
        nx.next(a);
        fetch_q(nx, w);
      }
      const uint32_t seg0 = t0 + i - cu.tile;
      finish_segment(seg0, seg0 + cu.s.n, w);
      if (last) break;
      cu = nx;
      start_segment();
    } else {
      cu.next(a);
    }
    stage = stage + 1 == NS ? 0 : stage + 1;
  }
  copy_wait<0>();
  if (n_shared == 0) return;
  __syncthreads();
  const Shared sh0 = shared[0], sh1 = shared[1];
  __syncthreads();
  if (sh0.last) join_shared(sh0);
  if (n_shared == 2 && sh1.last) join_shared(sh1);
}

template <class S>
cudaError_t launch_shape(const DecodeArgs &a, int grid, cudaStream_t s) {
  decode_kernel<S><<<grid, S::kThreads, S::kSmem, s>>>(a);
  return cudaGetLastError();
}
template <class S>
cudaError_t plan_shape(int *ctas_per_sm, int *tile) {
  *tile = S::kTile;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas_per_sm, decode_kernel<S>, S::kThreads, S::kSmem);
}

// Calls f with the shape of (d, e4m3, heads of a group).
template <class F>
cudaError_t with_shape(int d, bool e4m3, int group, F f) {
  const bool wide = group > 8;
  switch (d) {
    case 64:
      if (e4m3) return wide ? f(Shape<64, true, 16, 2, 8, 2, 1>{}) : f(Shape<64, true, 8, 2, 4, 2, 3>{});
      return wide ? f(Shape<64, false, 16, 2, 8, 2, 1>{}) : f(Shape<64, false, 8, 2, 4, 2, 3>{});
    case 128:
      if (e4m3) return wide ? f(Shape<128, true, 16, 2, 8, 2, 1>{}) : f(Shape<128, true, 8, 2, 4, 2, 2>{});
      return wide ? f(Shape<128, false, 16, 2, 8, 1, 1>{}) : f(Shape<128, false, 8, 2, 4, 1, 2>{});
    case 256:
      if (e4m3) return wide ? f(Shape<256, true, 16, 1, 8, 1, 1>{}) : f(Shape<256, true, 8, 2, 4, 1, 2>{});
      return wide ? f(Shape<256, false, 16, 1, 4, 1, 1>{}) : f(Shape<256, false, 8, 1, 4, 1, 2>{});
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int decode_group(int heads_per_kv) {
  const int n = (heads_per_kv + 15) / 16;
  return (heads_per_kv + n - 1) / n;
}

// With 2^k >= d > 2^(k - 1) and mul = floor(2^(31 + k) / d) + 1, mul * d exceeds
// 2^(31 + k) by at most d <= 2^k, so j * mul >> (31 + k) is j / d for every j < 2^31.
void decode_page_division(DecodeArgs *a) {
  const uint64_t d = (uint64_t)a->kv.page_size;
  int k = 0;
  while ((UINT64_C(1) << k) < d) ++k;
  a->page_mul = (uint32_t)((UINT64_C(1) << (31 + k)) / d + 1);
  a->page_shift = 31 + k;
  a->whole_pages = d % 16 == 0;
}

cudaError_t plan_paged_decode(int d, bool e4m3, int group, int *ctas_per_sm, int *tile) {
  return with_shape(d, e4m3, group, [&](auto s) { return plan_shape<decltype(s)>(ctas_per_sm, tile); });
}

cudaError_t launch_paged_decode(const DecodeArgs &a, int d, bool e4m3, int grid, cudaStream_t s) {
  return with_shape(d, e4m3, a.group, [&](auto sh) { return launch_shape<decltype(sh)>(a, grid, s); });
}

}  // namespace fp8moe
