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
// Measured, of the measured copy rate (6.70 TB/s), a few us of each being the
// launch, the search for the first tile, and the join:
//   64 sequences of up to 8192, 32 heads over 8, 128 elements, e4m3: 89.2 us, 6.01 TB/s, 90%
//   24 windows of up to 4096, 16 over 8, 256, bf16, capped scores:   61.2 us, 6.10 TB/s, 91%
//   8 of up to 4096, 16 over 16, 128, bf16:                          29.7 us, 5.31 TB/s, 79%
//   200 of up to 700, 24 over 6, 64, bf16, slopes:                   21.6 us, 3.52 TB/s, 53%
//   1 of 200001, 16 over 1, 128, e4m3:                               28.4 us, 1.86 TB/s, 28%
//   1 of 1000, 16 over 16, 128, bf16:                                 5.7 us, 1.43 TB/s, 21%
// The last ones are latency: the chain launch, length, page, rows, two products,
// join, and in groups of 16 heads the issue of the matrix instructions.
//
// Split.  A sequence's visible positions are cut into tiles of 16 or 32 keys, a
// segment is the tiles of one (sequence, group of up to 16 query heads that
// share a key/value head), and the list of all segments' tiles is cut evenly
// over the warps, whatever the lengths: every warp finds its piece from the
// lengths themselves.  In longer lists a segment counts a tile or two more, about
// what its start and end cost (64 sequences of up to 8192, e4m3, 89.4 us, not
// weighed 93.4; 200 of up to 700 21.6 and 24.3).  A warp writes the result of a
// segment that is all its own.  Of a piece at most the first and the last segment are shared
// with other warps; their parts (m, l, unnormalised output) stay in shared
// memory until all warps of the CTA are done, so the loop over tiles has no
// CTA-wide barrier, and are then joined.  A segment that several CTAs share
// goes to the workspace, and the CTA whose part came last joins it, in groups
// of 16 parts, then the groups.  The order of a join's sums is fixed by the
// parts' places, so results do not depend on the order of arrival.  No CTA
// waits for another.
//
// Few sequences.  Where every segment can have CTAs of its own, and no warp more
// than some tiles, what counts is the time before the first key and after the
// last.  Then a cluster of up to 8 CTAs takes one segment, or several clusters
// do: no list to search.  Each CTA of a cluster joins a share of the outputs, and
// every warp pushes its part of each share into that CTA's shared memory, so that
// one barrier of the cluster is all that stands between the last key and the
// cluster's result (one sequence of 1000, 32 heads over 8, bf16: 5.9 us; parts
// kept and pulled by the joining CTA, with a second barrier before the end, 7.9).
// Several clusters leave their results in the workspace, and the last CTA of
// those with the same share joins them (one sequence of 16000: 17.2 us, cut as a
// list 21.6).
//
// Tile.  Rows come through a ring of cp.async stages of each warp's own.
// S^T = K Q^T and O^T = V^T P^T run as mma.sync m16n8k16: 16 keys, then 16
// output columns, against 8 query heads (twice for groups of 9 to 16), so that
// few heads leave few lanes idle.  The order of the contraction over d and of
// the output columns is free, so both operands are read from shared memory as
// whole 16-byte pieces of a row: the order inside an instruction follows the
// lanes' pieces, not the row.  Weights pass from the scores' layout to the
// second product's by 8x8 transposes in registers (movmatrix).
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
//   s_j + log2(vs_j), so that they fit f16 whatever the scales.  Weights that are
//   small next to the largest may be all that a column has, and one f16 product
//   would lose those below 2^-21 of it (and hold the others to 11 bits), so what it
//   leaves, scaled by 2^12, is multiplied too and added apart: 22 bits together,
//   down to 2^-48 of the largest weight.  (The rest's product with scaled codes
//   instead: 64 x 8192 92.6 us, this way 89.3, one product alone 88.1.  Weights and
//   codes in bf16, which has no such limit: 103, most of it conversions.)
#include "common.cuh"
#include "kernels.h"
#include "paged_attn.h"

namespace fp8moe {

namespace {

constexpr int kJoin = 16;              // parts joined by one CTA
// Parts whose loads are in flight together: 2 take longer where parts are many (3
// sequences of up to 200000, 16 heads over one, e4m3: 40.9 -> 43.3 us), 16 by the
// size of their code in every call (32 of up to 4096, 16 heads: 27.5 -> 30.1).
constexpr int kBatch = 4;
constexpr int kWeighFrom = 4;          // tiles per warp from which on segments count more than their tiles
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLag = 8.f;            // log2 of the largest weight, before its scale
constexpr float kLagV = 4.f;           // the same with its scale
constexpr float kWeightBits = 11.f;    // e4m3: weights are scaled by 2^11, to 2^15 at most
constexpr float kRest = 0x1p12f;       // what f16 leaves of them (2^3 at most) by 2^12, to the same

// MH: query heads of a group at most; KM: 16-key steps of a warp's tile; NS:
// stages of a warp's ring; CTAS: that fit on an SM.  Tiles of 32 keys, 16 where
// more do not fit the registers (256 elements in bf16); two stages where rows are
// short (e4m3, 64 x 8192, 8 heads of 128 elements at most: 89.4 us, one 91.5), one
// where a tile is 16 KB, or 8 KB for 8 warps (32 x 4096, 16 heads: 27.5, two 29.8).
// 16 heads of 128 elements, and 256 elements in e4m3, take all 255 registers and
// spill (16 to 320 bytes a thread).
template <int D_, bool E4M3_, int MH_, int KM_, int kWarps_, int NS_, int CTAS_>
struct Shape {
  static constexpr int D = D_, MH = MH_, KM = KM_, NS = NS_, CTAS = CTAS_;
  static constexpr int kWarps = kWarps_, kThreads = 32 * kWarps;
  static constexpr int kKeys = 16 * KM;                          // keys of a tile
  static constexpr int kExtra = MH > 8 ? 2 : 1;                  // what a segment's start and end count for, in tiles
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
  // a warp's part of a shared segment, f32: the first of its piece has a place
  // of its own, the last one takes the place of the ring
  static constexpr int kPartRow = MH * (D + 4) * 4 <= NS * kStage ? D + 4 : D;
  static constexpr int kPart = MH * kPartRow * 4;
  static_assert(kPart <= NS * kStage, "a part fits the ring");
  static_assert(MH * D / 4 < 1024, "items of a segment");
  static_assert(kWarps <= 8, "a cluster has up to 32 warps");
  // shared memory: rings, first parts, (m, l) of both parts, their segments,
  // the segments shared with other CTAs, running sums of tiles
  static constexpr int kParts = kRing, kMl = kParts + kWarps * kPart, kSegs = kMl + 2 * kWarps * MH * 8;
  static constexpr int kShared = kSegs + 2 * kWarps * 32, kRuns = kShared + 2 * 32;
  static constexpr int kSmem = kRuns + (kThreads + kWarps) * 4;
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

// Two weights in 16 bits each, and what the pair leaves of them (f16: times 2^12).
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (F16) return pack_f16x2(a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2_rest(float a, float b, uint32_t high) {
  if (F16) {
    const float2 h = unpack_f16x2(high);
    return pack_f16x2((a - h.x) * kRest, (b - h.y) * kRest);
  }
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

// The even cut of W units over N warps: the first W % N take one more.
struct Cut {
  uint32_t each = 0, more = 0;
  Cut() = default;
  __device__ __forceinline__ Cut(uint32_t W, uint32_t N) : each(W / N), more(W % N) {}
  __device__ __forceinline__ uint32_t start(uint32_t warp) const { return each * warp + min(warp, more); }
  __device__ __forceinline__ uint32_t owner(uint32_t unit) const {
    const uint32_t big = more * (each + 1);
    return unit < big ? unit / (each + 1) : more + (unit - big) / each;
  }
};

// A segment that a warp holds a part of: its group of heads, its first unit and
// its number of tiles.
struct Segment {
  int b, ch, hg, n;
  uint32_t unit0;
  int valid;
  int unused[2];
};
// A segment that other CTAs hold parts of too: the CTA of the first part, the
// number of parts, and whether this CTA's part came last.
struct Shared {
  int b, ch, hg;
  int first, parts, last;
  int unused[2];
};
static_assert(sizeof(Segment) == 32 && sizeof(Shared) == 32, "as laid out in Shape");

// Adds N parts (m, l, output piece) to (mm, ll, v), under their common maximum top.
template <int N>
__device__ __forceinline__ void add_parts(float &mm, float &ll, float4 &v, float top, const float2 (&st)[N],
                                          const float4 (&x)[N]) {
  const float f0 = rescale(mm, top);
  ll *= f0;
  v = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
  mm = top;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float f = rescale(st[i].x, top);
    ll = fmaf(f, st[i].y, ll);
    v = make_float4(fmaf(f, x[i].x, v.x), fmaf(f, x[i].y, v.y), fmaf(f, x[i].z, v.z), fmaf(f, x[i].w, v.w));
  }
}

// CLUSTER: a.splits clusters of a.cluster CTAs per segment, else the list of tiles.
template <class S, bool CLUSTER>
__global__ void __launch_bounds__(S::kThreads, S::CTAS) decode_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int D = S::D, MH = S::MH, NT = S::NT, NS = S::NS, EV = S::EV, KM = S::KM;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kKeys = S::kKeys;
  constexpr bool Q8 = S::E4M3;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;  // row and column of the matrix instructions
  float2 *ml = reinterpret_cast<float2 *>(smem + S::kMl);          // [2 * warp + which][MH]
  Segment *segs = reinterpret_cast<Segment *>(smem + S::kSegs);    // [2 * warp + which]
  Shared *shared = reinterpret_cast<Shared *>(smem + S::kShared);  // [2]
  uint32_t *runs = reinterpret_cast<uint32_t *>(smem + S::kRuns);  // [kThreads], then a sum per warp
  const int G = a.n_heads / a.n_kv;
  pdl_wait();
  pdl_trigger();

  // ---- the W tiles of all sequences: running sums over runs of `per` sequences
  const auto count = [&](int b) {
    const int len = a.lens[b];
    if (len < 0 || len > a.capacity) set_error(a.err, DEV_ERR_BOUNDS);
    return (uint32_t)(span_of<kKeys>(a, b).n * a.n_groups);
  };
  const auto scan = [&](uint32_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    return v;
  };
  // The queries of a segment as a lane holds them: heads g + 8n.  The first
  // segment's are asked for ahead of its pages and rows, whose latency covers theirs.
  uint4 qw[NT][D / 32];
  const auto load_q = [&](int b, int ch, int hg) {
    const int in_kv = hg * a.group, heads = min(a.group, G - in_kv);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = g + 8 * n;
      const __nv_bfloat16 *qp = a.q + (int64_t)b * a.q_stride + (int64_t)(ch * G + in_kv + h) * D;
#pragma unroll
      for (int s = 0; s < D / 32; ++s) {
        // bf16: piece c + 4s of 8 elements; e4m3: halves of piece c + 4 (s / 2) of 16
        const int at = Q8 ? (c + 4 * (s / 2)) * 16 + 8 * (s & 1) : (c + 4 * s) * 8;
        qw[n][s] = h < heads ? *reinterpret_cast<const uint4 *>(qp + at) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  uint32_t unit = 0;
  int my_part = 0;          // of a cluster's segment
  int left = 0, extra = 0;  // tiles and units of this warp's piece that are left
  Cut cut;
  Cursor<kKeys> cu{};
  if constexpr (CLUSTER) {  // ---- the tiles of a segment, cut over the warps of its clusters
    // (waited for before anything is pushed to a CTA that may not have begun)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int seg = blockIdx.x / (a.splits * a.cluster), vh = seg % a.n_groups;
    cu.b = seg / a.n_groups;
    cu.ch = vh / a.groups_per_kv;
    cu.hg = vh - cu.ch * a.groups_per_kv;
    load_q(cu.b, cu.ch, cu.hg);
    count(cu.b);
    cu.s = span_of<kKeys>(a, cu.b);
    const Cut tiles(cu.s.n, a.splits * a.cluster * kWarps);
    const int me = (blockIdx.x - seg * a.splits * a.cluster) * kWarps + warp;
    cu.tile = (int)tiles.start(me);
    left = (int)tiles.start(me + 1) - cu.tile;
    my_part = me % (a.cluster * kWarps);
    unit = cu.tile;
  } else {
    const int per = a.B <= kThreads ? 1 : (a.B + kThreads - 1) / kThreads;
    uint32_t W;
    if (a.B <= 32) {  // every warp for itself, to the same result
      const uint32_t incl = scan(lane < a.B ? count(lane) : 0);
      W = __shfl_sync(0xffffffffu, incl, 31);
      runs[lane] = incl;
      __syncwarp();
    } else {
      const int b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
      uint32_t mine = 0;
      for (int b = b0; b < b1; ++b) mine += count(b);
      uint32_t incl = scan(mine);
      if (lane == 31) runs[kThreads + warp] = incl;
      __syncthreads();
      W = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) incl += runs[kThreads + w];
        W += runs[kThreads + w];
      }
      runs[threadIdx.x] = incl;
      __syncthreads();
    }
    // ---- this warp's piece.  A segment has a unit for each tile and `extra`
    // ones after them.
    const uint32_t n_warps = min(W, gridDim.x * kWarps), me = blockIdx.x * kWarps + warp;
    if (blockIdx.x * kWarps >= n_warps) return;
    extra = W >= kWeighFrom * kWarps * gridDim.x ? S::kExtra : 0;
    const auto units_of = [&](uint32_t tiles, int segments) { return tiles + (uint32_t)(extra * segments); };
    cut = Cut(units_of(W, a.n_groups * a.B), n_warps);
    unit = cut.start(me);
    left = me < n_warps ? (int)(cut.start(me + 1) - unit) : 0;  // units
    if (left > 0) {  // the sequence of the first unit, and the place within it
      int run = 0;
      for (int base = 0;; base += 32) {
        const int r = base + lane, end = min((r + 1) * per, a.B);
        const bool beyond = r * per >= a.B || units_of(runs[min(r, kThreads - 1)], a.n_groups * end) > unit;
        const uint32_t found = __ballot_sync(0xffffffffu, beyond);
        if (found != 0) {
          run = base + __ffs((int)found) - 1;
          break;
        }
      }
      uint32_t before = run > 0 ? runs[run - 1] : 0;  // tiles of the sequences before cu.b
      cu.b = run * per;
      if (per > 1) {
        const int end = min(cu.b + per, a.B);
        for (int base = cu.b;; base += 32) {
          const uint32_t n = base + lane < end ? (uint32_t)(span_of<kKeys>(a, base + lane).n * a.n_groups) : 0;
          const uint32_t incl = scan(n);
          const uint32_t found = __ballot_sync(
              0xffffffffu, base + lane >= end - 1 ||
                               units_of(before + incl, a.n_groups * (base + lane + 1)) > unit);
          if (found != 0) {
            const int at = __ffs((int)found) - 1;
            cu.b = base + at;
            before += __shfl_sync(0xffffffffu, incl - n, at);
            break;
          }
          before += __shfl_sync(0xffffffffu, incl, 31);
        }
      }
      cu.s = span_of<kKeys>(a, cu.b);
      const uint32_t r = unit - units_of(before, a.n_groups * cu.b);
      const int vh = (int)(r / (cu.s.n + extra));
      cu.tile = (int)r - vh * (cu.s.n + extra);
      cu.ch = vh / a.groups_per_kv;
      cu.hg = vh - cu.ch * a.groups_per_kv;
      if (cu.tile >= cu.s.n) {  // it begins with a segment's extra units
        const int skip = cu.s.n + extra - cu.tile;
        left -= skip;
        unit += skip;
        cu.tile = cu.s.n - 1;
        if (left > 0) cu.next(a);
      }
    }
  }

  // ---- loads: the rows of a warp's keys, NS stages ahead of their use
  constexpr int kRowsAtOnce = 32 / S::kPieces;  // rows of one copy instruction
  constexpr uint32_t kAll = kKeys == 32 ? 0xffffffffu : (1u << kKeys) - 1;
  const uint32_t ring = smem_addr(smem) + warp * (NS * S::kStage);
  const int my_key = lane & (kKeys - 1), my_row = lane / S::kPieces, my_piece = lane % S::kPieces;
  const int64_t my_off = my_row * a.kv.slot_stride + my_piece * 16;
  const int64_t row_step = kRowsAtOnce * a.kv.slot_stride;
  Cursor<kKeys> ld = cu;
  int ld_left = left;
  int32_t page = -1;          // page of this lane's key in the next tile to load
  int64_t row = 0, srow = 0;  // offsets of its row and its scales
  uint32_t on = 0;            // keys of the tile that are loaded
  auto page_index = [&](int j) { return (int)(((uint64_t)(uint32_t)j * a.page_mul) >> a.page_shift); };
  auto fetch_page = [&]() {
    if (ld_left <= 0) return;
    const int j = (ld.s.first + ld.tile) * kKeys + my_key;
    page = -1;
    if (j >= ld.s.lo && j < ld.s.hi) page = a.table[ld.b * a.table_stride + page_index(j)];
  };
  // brings the queries of a segment near, ahead of its first tile
  const auto fetch_q = [&](const Cursor<kKeys> &k) {
    const int in_kv = k.hg * a.group, heads = min(a.group, G - in_kv);
    const __nv_bfloat16 *q = a.q + (int64_t)k.b * a.q_stride + (int64_t)(k.ch * G + in_kv) * D;
    for (int i = lane * 64; i < heads * D; i += 32 * 64) asm volatile("prefetch.global.L1 [%0];" ::"l"(q + i));
  };
  auto load_half = [&](int stage, bool is_v) {
    if (ld_left > 0 && ld.s.lo < ld.s.hi) {
      const uint32_t dst = ring + stage * S::kStage + (is_v ? S::kHalfTile : 0);
      if (!is_v) {  // where the keys lie; the same for their value rows
        const int j = (ld.s.first + ld.tile) * kKeys + my_key;
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
    if (is_v && ld_left > 0) {
      --ld_left;
      if (ld.tile == ld.s.n - 1) ld_left -= extra;
      if (ld_left > 0) {
        ld.next(a);
        fetch_page();
        if (ld.tile == 0) fetch_q(ld);
      }
    }
  };
  if (!CLUSTER && left > 0) load_q(cu.b, cu.ch, cu.hg);
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
  auto start_segment = [&]() {
    const int in_kv = cu.hg * a.group;
    const int heads = min(a.group, G - in_kv), head0 = cu.ch * G + in_kv;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
      const auto &w = qw[n];
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
    const int base = (cu.s.first + cu.tile) * kKeys;
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
          high |= top > mv[n][u] + kLagV;
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
          p_lo[t][n][u] = transpose8(pack2_rest<Q8>(p[2 * u], p[2 * u + 1], hi));
        }
      }
    }
  };
  auto add_values = [&](int stage, const uint32_t (&p_hi)[KM][NT][2], const uint32_t (&p_lo)[KM][NT][2]) {
    const uint32_t vb = ring + stage * S::kStage + S::kHalfTile;
    const auto load = [&](uint4 (&v)[4], int t, int h) {
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
    };
    if constexpr (!Q8) {
#pragma unroll
      for (int t = 0; t < KM; ++t)
#pragma unroll
        for (int h = 0; h < S::H; ++h) {
          uint4 v[4];
          load(v, t, h);
#pragma unroll
          for (int w = 0; w < 4; ++w) {  // columns 2w, 2w + 1 of the piece, keys paired
            const uint32_t v0 = u4_word(v[0], w), v1 = u4_word(v[1], w), v2 = u4_word(v[2], w),
                           v3 = u4_word(v[3], w);
            const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
            const uint32_t a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816<false>(o[n][4 * h + w], a0, a1, a2, a3, p_hi[t][n][0], p_hi[t][n][1]);
              mma16816<false>(o[n][4 * h + w], a0, a1, a2, a3, p_lo[t][n][0], p_lo[t][n][1]);
            }
          }
        }
    } else {
#pragma unroll
      for (int h = 0; h < S::H; ++h) {
        uint4 v[KM][4];
#pragma unroll
        for (int t = 0; t < KM; ++t) load(v[t], t, h);
#pragma unroll
        for (int w = 0; w < EV / 4; ++w)
#pragma unroll
          for (int u = 0; u < 2; ++u) {  // columns 4w + 2u, + 1
            float rest[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) rest[n][0] = rest[n][1] = rest[n][2] = rest[n][3] = 0.f;
#pragma unroll
            for (int t = 0; t < KM; ++t) {
              const uint32_t v0 = u4_word(v[t][0], w), v1 = u4_word(v[t][1], w), v2 = u4_word(v[t][2], w),
                             v3 = u4_word(v[t][3], w);
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(__byte_perm(v0, v1, u ? 0x7362 : 0x5140), a0, a1);
              e4m3x4_to_f16(__byte_perm(v2, v3, u ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma16816<true>(o[n][EV / 2 * h + 2 * w + u], a0, a1, a2, a3, p_hi[t][n][0], p_hi[t][n][1]);
                mma16816<true>(rest[n], a0, a1, a2, a3, p_lo[t][n][0], p_lo[t][n][1]);
              }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float &to = o[n][EV / 2 * h + 2 * w + u][i];
                to = fmaf(rest[n][i], 1.f / kRest, to);
              }
          }
      }
    }
  };

  // ---- end of a segment, or of this warp's part of it
  // Sums over the lanes of a column, and the factor of the outputs under m.
  const auto total = [&](int n, int u) {
    float sum = l[n][u];
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    return sum;
  };
  const auto under_m = [&](int n, int u) {
    return Q8 && m[n][u] != -INFINITY && mv[n][u] != -INFINITY ? ex2(mv[n][u] - m[n][u] - kWeightBits) : 1.f;
  };
  const auto lse_of = [](float mm, float ll) { return (mm + log2f(ll)) * kLn2; };
  auto write_whole = [&]() {
    const int in_kv = cu.hg * a.group, heads = min(a.group, G - in_kv);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float ll = total(n, u), f = under_m(n, u) * (ll == 0.f ? 0.f : 1.f / ll);
        const int h = 8 * n + 2 * c + u;
        if (h >= heads) continue;
        const int64_t bh = (int64_t)cu.b * a.n_heads + cu.ch * G + in_kv + h;
#pragma unroll
        for (int hh = 0; hh < S::H; ++hh)
#pragma unroll
          for (int jj = 0; jj < EV / 8; ++jj) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float *x = o[n][EV / 2 * hh + 4 * jj + i];
              w[i] = pack2<false>(x[u] * f, x[2 + u] * f);
            }
            *reinterpret_cast<uint4 *>(a.out + bh * D + (g + 8 * hh) * EV + 8 * jj) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        if (g == 0 && a.lse) a.lse[bh] = lse_of(m[n][u], ll);
      }
  };
  // How a cluster shares a segment's float4 items out: `share` to a CTA, which
  // touch at most `span` heads.
  struct Shares {
    int items, share, span;
    uint32_t mul;  // the CTA of item i is i * mul >> 20 (items < 1024)
  };
  const auto shares_of = [&](int heads) {
    Shares z;
    z.items = heads * (D / 4);
    z.share = z.items / a.cluster;
    z.span = z.share / (D / 4) + (z.share % (D / 4) == 0 ? 0 : 2);
    z.mul = ((1u << 20) * a.cluster + z.items - 1) / z.items;
    return z;
  };
  const auto in_cta = [&](int byte, int rank) {  // a place in the shared memory of a CTA of the cluster
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(smem) + byte), "r"(rank));
    return at;
  };
  auto push_part = [&]() {
    const int heads = min(a.group, G - cu.hg * a.group);
    const Shares z = shares_of(heads);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float ll = total(n, u), f = under_m(n, u);
        const int h = 8 * n + 2 * c + u;
        if (h >= heads) continue;
#pragma unroll
        for (int hh = 0; hh < S::H; ++hh)
#pragma unroll
          for (int jj = 0; jj < EV / 4; ++jj) {
            const int i = h * (D / 4) + (g + 8 * hh) * (EV / 4) + jj, rank = (int)((i * z.mul) >> 20);
            const float *x = o[n][EV / 2 * hh + 2 * jj], *y = o[n][EV / 2 * hh + 2 * jj + 1];
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                             in_cta(S::kParts + (my_part * z.share + i - rank * z.share) * 16, rank)),
                         "f"(x[u] * f), "f"(x[2 + u] * f), "f"(y[u] * f), "f"(y[2 + u] * f)
                         : "memory");
          }
        if (g == 0) {  // (m, l) to all that share the head
          const int last = (int)(((h * (D / 4) + D / 4 - 1) * z.mul) >> 20);
          for (int rank = (int)((h * (D / 4) * z.mul) >> 20); rank <= last; ++rank)
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(
                             in_cta(S::kMl + (my_part * z.span + h - rank * z.share / (D / 4)) * 8, rank)),
                         "f"(m[n][u]), "f"(ll)
                         : "memory");
        }
      }
  };
  // Where part `which` (0: the first of a piece, 1: the last) of a warp lies.
  const auto part_at = [&](int w, int which) {
    return reinterpret_cast<float *>(smem + (which == 0 ? S::kParts + w * S::kPart : w * (NS * S::kStage)));
  };
  auto keep_part = [&](int which, uint32_t unit0) {
    const int heads = min(a.group, G - cu.hg * a.group);
    float *const to = part_at(warp, which);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float ll = total(n, u), f = under_m(n, u);
        const int h = 8 * n + 2 * c + u;
        if (h >= heads) continue;
#pragma unroll
        for (int hh = 0; hh < S::H; ++hh)
#pragma unroll
          for (int jj = 0; jj < EV / 4; ++jj) {
            const float *x = o[n][EV / 2 * hh + 2 * jj], *y = o[n][EV / 2 * hh + 2 * jj + 1];
            *reinterpret_cast<float4 *>(to + h * S::kPartRow + (g + 8 * hh) * EV + 4 * jj) =
                make_float4(x[u] * f, x[2 + u] * f, y[u] * f, y[2 + u] * f);
          }
        if (g == 0) ml[(2 * warp + which) * MH + h] = make_float2(m[n][u], ll);
      }
    if (lane == 0) segs[2 * warp + which] = Segment{cu.b, cu.ch, cu.hg, cu.s.n, unit0, 1, {0, 0}};
  };

  if (lane < 2) segs[2 * warp + lane].valid = 0;
  __syncwarp();
  int stage = 0;
  while (left > 0) {  // the parts of segments in this piece
    const int from = cu.tile, to = min(cu.s.n, from + left);
    const bool busy = cu.s.lo < cu.s.hi;
    start_segment();
    for (; cu.tile < to; ++cu.tile) {
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
      stage = stage + 1 == NS ? 0 : stage + 1;
    }
    const uint32_t unit0 = unit - from;
    unit += to - from + extra;
    left -= to - from + (to == cu.s.n ? extra : 0);
    if (from == 0 && to == cu.s.n) {
      write_whole();
    } else {
      const int which = left > 0 ? 0 : 1;
      if constexpr (CLUSTER) {
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        push_part();
      } else {
        if (which == 1) {
          copy_wait<0>();
          __syncwarp();  // the ring is free
        }
        keep_part(which, unit0);
      }
    }
    --cu.tile;
    if (left > 0) {
      cu.next(a);
      load_q(cu.b, cu.ch, cu.hg);
    }
  }
  // Counts a part that all threads have written; true for the last.
  const auto arrive = [&](int *counter, int n) {
    int before;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    if (before == n - 1) *counter = 0;  // for the next call
    return before == n - 1;
  };
  copy_wait<0>();
  if constexpr (CLUSTER) {
    // the segment's first warps have a part each
    const int warps = a.cluster * kWarps, clusters = min((cu.s.n + warps - 1) / warps, a.splits);
    const int cluster_at = blockIdx.x / a.cluster, nth = cluster_at % a.splits;
    const int parts = min(max(cu.s.n - nth * warps, 0), warps);
    const bool whole = cu.s.n == 1;
    __syncwarp();
    // those without a part, or with the whole, have not waited yet
    if (my_part >= parts || whole) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (parts == 0 || whole) return;
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const int in_kv = cu.hg * a.group, heads = min(a.group, G - in_kv);
    const int64_t head0 = (int64_t)cu.b * a.n_heads + cu.ch * G + in_kv;
    const Shares z = shares_of(heads);
    const int rank = blockIdx.x % a.cluster, i0 = rank * z.share;
    // Joins n parts of this CTA's items with `lanes` (a power of two) neighbouring
    // lanes per item, a part each at a time; load(part, head, item of the segment,
    // (m, l), piece), store(head, item of the head, piece, m, l).
    const auto join = [&](int n, const auto &load, const auto &store) {
      int lanes = 1;
      while (2 * lanes * z.share <= kThreads && 2 * lanes <= min(32, n)) lanes *= 2;
      const int sub = threadIdx.x & (lanes - 1);
#pragma unroll 1
      for (int base = 0; base < z.share; base += kThreads / lanes) {
        const int j = base + threadIdx.x / lanes, i = i0 + min(j, z.share - 1);
        const int h = i / (D / 4), it = i % (D / 4);
        float mm = -INFINITY, ll = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int p = sub; p < n; p += 4 * lanes) {
          float2 st[4];
          float4 x[4];
          float top = mm;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            st[q] = make_float2(-INFINITY, 0.f);
            x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p + q * lanes < n) load(p + q * lanes, h, i, st[q], x[q]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) top = fmaxf(top, st[q].x);
          add_parts<4>(mm, ll, v, top, st, x);
        }
        // all five steps, without branches, so that the sums overlap
        float top = mm;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float t = __shfl_xor_sync(0xffffffffu, top, o);
          top = o < lanes ? fmaxf(top, t) : top;
        }
        const float f = rescale(mm, top);
        ll *= f;
        v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float t = __shfl_xor_sync(0xffffffffu, ll, o), tx = __shfl_xor_sync(0xffffffffu, v.x, o),
                      ty = __shfl_xor_sync(0xffffffffu, v.y, o), tz = __shfl_xor_sync(0xffffffffu, v.z, o),
                      tw = __shfl_xor_sync(0xffffffffu, v.w, o);
          if (o < lanes) {
            ll += t;
            v = make_float4(v.x + tx, v.y + ty, v.z + tz, v.w + tw);
          }
        }
        if (sub == 0 && j < z.share) store(h, it, i, v, top, ll);
      }
    };
    const auto write = [&](int h, int it, int, float4 v, float mm, float ll) {
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
      uint2 w;
      w.x = pack2<false>(v.x * inv, v.y * inv);
      w.y = pack2<false>(v.z * inv, v.w * inv);
      *reinterpret_cast<uint2 *>(a.out + (head0 + h) * D + 4 * it) = w;
      if (it == 0 && a.lse) a.lse[head0 + h] = lse_of(mm, ll);
    };
    const float4 *x_at = reinterpret_cast<const float4 *>(smem + S::kParts) - i0;
    const float2 *ml_at = ml - i0 / (D / 4);
    const auto pushed = [&](int p, int h, int i, float2 &st, float4 &x) {
      st = ml_at[p * z.span + h];
      x = x_at[p * z.share + i];
    };
    if (clusters == 1) {
      join(parts, pushed, write);
      return;
    }
    // Several clusters: each CTA leaves what it joined in the workspace, the last
    // of those with the same share joins them.
    float4 *const part = reinterpret_cast<float4 *>(a.part);    // [cluster][group * D / 4]
    float2 *const part_ml = reinterpret_cast<float2 *>(a.part_ml);  // [CTA][group]
    const int64_t row = (int64_t)a.group * (D / 4);
    join(parts, pushed, [&](int h, int it, int i, float4 v, float mm, float ll) {
      part[cluster_at * row + i] = v;
      if (it == 0 || i == i0) part_ml[(int64_t)blockIdx.x * a.group + h] = make_float2(mm, ll);
    });
    __syncthreads();
    if (threadIdx.x == 0) shared[0].last = arrive(a.counters + cluster_at / a.splits * a.cluster + rank, clusters);
    __syncthreads();
    if (!shared[0].last) return;
    const int64_t first = cluster_at - nth;
    join(clusters, [&](int p, int h, int i, float2 &st, float4 &x) {
      st = __ldcg(part_ml + ((first + p) * a.cluster + rank) * a.group + h);
      x = __ldcg(part + (first + p) * row + i);
    }, write);
    return;
  }
  __syncthreads();

  // ---- the CTA's shared segments
  float4 *part = reinterpret_cast<float4 *>(a.part);
  float2 *part_ml = reinterpret_cast<float2 *>(a.part_ml);
  // Outputs are handled as float4 items: item i of a head is elements 4i .. 4i + 3.
  const auto write_out = [&](int b, int head, int item, float4 v, float mm, float ll) {
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const int64_t bh = (int64_t)b * a.n_heads + head;
    uint2 w;
    w.x = pack2<false>(v.x * inv, v.y * inv);
    w.y = pack2<false>(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2 *>(a.out + bh * D + 4 * item) = w;
    if (item == 0 && a.lse) a.lse[bh] = lse_of(mm, ll);
  };
  // A CTA's slots of the workspace: 0 for a segment that began in another CTA,
  // 1 for one that begins here.
  const auto slot_of = [&](int first, int nth) { return 2 * (first + nth) + (nth == 0 ? 1 : 0); };
  // Warps take 32 items at a time, the next segment's after this one's.
  int n_shared = 0, i0 = threadIdx.x;
  const uint32_t valid = __ballot_sync(0xffffffffu, lane < 2 * kWarps && segs[lane & (2 * kWarps - 1)].valid);
  for (uint32_t rest = valid; rest != 0;) {
    const Segment sg = segs[__ffs((int)rest) - 1];
    // the warps' parts of this segment
    const uint32_t same = rest & __ballot_sync(0xffffffffu, segs[lane & (2 * kWarps - 1)].unit0 == sg.unit0);
    rest &= ~same;
    const int in_kv = sg.hg * a.group, heads = min(a.group, G - in_kv);
    const int head0 = sg.ch * G + in_kv, items = heads * (D / 4);
    const int first = (int)(cut.owner(sg.unit0) / kWarps);
    const int parts = (int)(cut.owner(sg.unit0 + sg.n - 1) / kWarps) - first + 1;
    const int mine = slot_of(first, blockIdx.x - first);
#pragma unroll 1
    for (int i = i0; i < items; i += kThreads) {
      const int h = i / (D / 4), it = i % (D / 4);
      float mm = -INFINITY, ll = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (uint32_t set = same; set != 0;) {  // four at a time
        float2 st[4];
        float4 x[4];
        float top = mm;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int p = __ffs((int)set) - 1;
          st[q] = make_float2(-INFINITY, 0.f);
          x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (set != 0) {
            st[q] = ml[p * MH + h];
            x[q] = *reinterpret_cast<const float4 *>(part_at(p / 2, p & 1) + h * S::kPartRow + 4 * it);
          }
          set &= set - 1;
          top = fmaxf(top, st[q].x);
        }
        add_parts<4>(mm, ll, v, top, st, x);
      }
      if (parts == 1) {
        write_out(sg.b, head0 + h, it, v, mm, ll);
      } else {
        part[((int64_t)mine * a.group + h) * (D / 4) + it] = v;
        if (it == 0) part_ml[(int64_t)mine * a.group + h] = make_float2(mm, ll);
      }
    }
    i0 = (i0 - ((items + 31) & ~31)) & (kThreads - 1);
    if (parts > 1) {
      if (threadIdx.x == 0) shared[n_shared] = Shared{sg.b, sg.ch, sg.hg, first, parts, 0, {0, 0}};
      ++n_shared;
    }
  }
  if (n_shared == 0) return;
  // Counters: a CTA is the first of at most one shared segment and a later one
  // of at most one other, so three arrays by CTA do.
  __syncthreads();
  if (lane == 0 && warp < n_shared) {
    const int first = shared[warp].first, grp = ((int)blockIdx.x - first) / kJoin;
    shared[warp].last = arrive(a.counters + (grp == 0 ? 0 : a.max_ctas) + first + grp * kJoin,
                               min(kJoin, shared[warp].parts - grp * kJoin));
  }
  __syncthreads();
  for (int i = 0; i < n_shared; ++i) {
    const Shared sh = shared[i];
    if (!sh.last) continue;
    // this CTA's group of the segment's parts, then, if that was the last
    // group, the groups
    const int first = sh.first, in_kv = sh.hg * a.group, heads = min(a.group, G - in_kv);
    const int head0 = sh.ch * G + in_kv, items = heads * (D / 4);
    const int groups = (sh.parts + kJoin - 1) / kJoin;
    int p0 = ((int)blockIdx.x - first) / kJoin * kJoin, step = 1, n = min(kJoin, sh.parts - p0);
    bool final = groups == 1;
    for (;;) {  // n parts, every `step`-th from p0 on
#pragma unroll 1
      for (int j = threadIdx.x; j < items; j += kThreads) {
        const int h = j / (D / 4), it = j % (D / 4);
        float mm = -INFINITY, ll = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int p = 0; p < n; p += kBatch) {
          float2 st[kBatch];
          float4 x[kBatch];
#pragma unroll
          for (int q = 0; q < kBatch; ++q) {
            st[q] = make_float2(-INFINITY, 0.f);
            x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p + q < n) {
              const int64_t at = (int64_t)slot_of(first, p0 + (p + q) * step) * a.group + h;
              st[q] = __ldcg(part_ml + at);
              x[q] = __ldcg(part + at * (D / 4) + it);
            }
          }
          float top = mm;
#pragma unroll
          for (int q = 0; q < kBatch; ++q) top = fmaxf(top, st[q].x);
          add_parts<kBatch>(mm, ll, v, top, st, x);
        }
        if (final) {
          write_out(sh.b, head0 + h, it, v, mm, ll);
        } else {  // in place of the group's first part, which only this thread has read ..
          part[((int64_t)slot_of(first, p0) * a.group + h) * (D / 4) + it] = v;
          if (it == 0) ml[h] = make_float2(mm, ll);  // .. except for its statistics
        }
      }
      if (final) break;
      __syncthreads();
      for (int h = threadIdx.x; h < heads; h += kThreads)
        part_ml[(int64_t)slot_of(first, p0) * a.group + h] = ml[h];
      __syncthreads();
      if (threadIdx.x == 0) shared[i].last = arrive(a.counters + 2 * a.max_ctas + first, groups);
      __syncthreads();
      if (!shared[i].last) break;
      p0 = 0;
      step = kJoin;
      n = groups;
      final = true;
    }
  }
}

template <class S>
cudaLaunchConfig_t launch_config(const DecodeArgs &a, int grid, cudaStream_t s, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  return cfg;
}
template <class S, bool CLUSTER>
cudaError_t launch_shape(const DecodeArgs &a, int grid, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = launch_config<S>(a, grid, s, attr);
  return cudaLaunchKernelEx(&cfg, decode_kernel<S, CLUSTER>, a);
}
template <class S>
cudaError_t plan_shape(int *ctas_per_sm, int *tile, int *warps, int (&clusters)[4]) {
  *tile = S::kKeys;
  *warps = S::kWarps;
  int n[2] = {0, 0};
  const auto plan = [](auto kernel, int *fit) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(fit, kernel, S::kThreads, S::kSmem);
  };
  cudaError_t e = plan(decode_kernel<S, false>, &n[0]);
  if (e == cudaSuccess) e = plan(decode_kernel<S, true>, &n[1]);
  *ctas_per_sm = n[0] < n[1] ? n[0] : n[1];
  for (int i = 1; i < 4 && e == cudaSuccess; ++i) {
    DecodeArgs a = {};
    a.cluster = 1 << i;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = launch_config<S>(a, 1 << i, nullptr, attr);
    e = cudaOccupancyMaxActiveClusters(&clusters[i], decode_kernel<S, true>, &cfg);
  }
  return e;
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
      if (e4m3) return wide ? f(Shape<128, true, 16, 2, 8, 1, 1>{}) : f(Shape<128, true, 8, 2, 4, 2, 2>{});
      return wide ? f(Shape<128, false, 16, 2, 8, 1, 1>{}) : f(Shape<128, false, 8, 2, 4, 1, 2>{});
    case 256:
      if (e4m3) return f(Shape<256, true, 8, 2, 4, 1, 2>{});
      return f(Shape<256, false, 8, 1, 4, 1, 2>{});
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// Up to 16 heads at a time: in long lists a second pass over the rows costs more
// than wider steps (16 heads of 128 elements, 32 sequences of up to 4096 tokens, 4
// key/value heads: e4m3 27.5 us, against 31.3 in groups of 8; bf16 31.3 against 35.6).
// 16 heads of 256 elements would take 128 registers for the outputs and 64 for the
// queries, which leaves too few for a tile; groups of 8 read their rows from L2 the
// second time (32 sequences of up to 2048: e4m3 35.1 us, bf16 40.0).
int decode_group(int heads_per_kv, int d, bool narrow) {
  const int most = narrow || d == 256 ? 8 : 16, n = (heads_per_kv + most - 1) / most;
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

cudaError_t plan_paged_decode(int d, bool e4m3, int group, int *ctas_per_sm, int *tile, int *warps,
                              int (&clusters)[4]) {
  return with_shape(d, e4m3, group,
                    [&](auto s) { return plan_shape<decltype(s)>(ctas_per_sm, tile, warps, clusters); });
}

cudaError_t launch_paged_decode(const DecodeArgs &a, int d, bool e4m3, int grid, cudaStream_t s) {
  return with_shape(d, e4m3, a.group, [&](auto sh) {
    return a.cluster > 0 ? launch_shape<decltype(sh), true>(a, grid, s)
                         : launch_shape<decltype(sh), false>(a, grid, s);
  });
}

}  // namespace fp8moe
