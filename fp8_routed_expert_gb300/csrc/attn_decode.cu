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
// Split.  A sequence's visible positions are cut into tiles of 64, a segment
// is the tiles of one (sequence, group of up to 16 query heads that share a
// key/value head), and the list of all segments' tiles is cut evenly over the
// CTAs, whatever the lengths: every CTA finds its piece from the lengths
// themselves.  A CTA that holds a segment's whole list writes its result; the
// pieces of a segment that several CTAs share go to the workspace as (m, l,
// unnormalised output) and the last CTA to arrive joins them, in groups of 16
// pieces, then the groups.  The order of a join's sums is fixed by the
// pieces' places, so results do not depend on the order of arrival.  No CTA
// waits for another.
//
// Tile.  Each of a CTA's four warps takes 16 of a tile's 64 keys through its
// own ring of cp.async stages and keeps its own (m, l, output), so the loop
// has no CTA-wide barrier.  S = Q K^T and O = P V run as mma.sync m16n8k16
// with the query heads as the 16 rows.  The order of the contraction and of
// the output columns is free, so both operands are read from shared memory as
// whole 16-byte pieces of a row: element order inside an instruction follows
// the lanes' pieces, not the row.  A score's accumulator is in the layout the
// next product wants its weights in.
//   bf16 rows: weights need more than bf16's 8 bits, so they are split into a
//   high and a low bf16 part (16 bits together).  With at most 8 heads the low
//   parts are the rows 8-15 that would otherwise be padding; with 9 to 16
//   heads they are a second product.
//   e4m3 rows: codes become f16 (exact), q becomes f16 with a power-of-two
//   shift per head that puts its largest value at 2^14 (exact down to 2^-28 of
//   it), a key's scale multiplies its score, and a value's scale joins the
//   exponent: weights e^(s_j - m') vs_j with a second running maximum m' of
//   s_j + log2(vs_j), so that they fit f16 whatever the scales.  Weights are
//   then at most 2^15 and kept to f16's 11 bits, with low parts for up to 8
//   heads as above.
#include "common.cuh"
#include "paged_attn.h"

namespace fp8moe {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 16;              // keys of a warp's tile
constexpr int kTile = kWarps * kKeys;  // keys of a CTA's tile
constexpr int kJoin = 16;              // pieces joined at a time
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kWeightBits = 15.f;    // e4m3: weights are scaled by 2^15

template <int D_, bool E4M3_, int MH_, int NS_>
struct Shape {
  static constexpr int D = D_, MH = MH_, NS = NS_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
  static constexpr int kPieces = kRowBytes / 16;              // 16-byte pieces of a row
  static constexpr int kHalfTile = kKeys * kRowBytes;         // a warp's K or V rows
  static constexpr int kStage = 2 * kHalfTile + (E4M3 ? 8 * kKeys : 0);
  static constexpr int kRing = kWarps * NS * kStage;
  // values per lane and value row: a 16-byte piece, 8 bytes for the shortest row
  static constexpr int EV = E4M3 && D > 64 ? 16 : 8;
  static constexpr int H = D / (8 * EV);
  static constexpr int kMerge = kWarps * MH * D * 4;          // f32 outputs of the warps
  static constexpr int kSmem = kRing + kMerge + kWarps * MH * 8 + 64;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// 16 / 4 bytes to shared memory, zeros where !on.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
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
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// Two weights of neighbouring keys as the high part, and what it leaves.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (F16) return pack_f16x2(a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2_rest(float a, float b, uint32_t high) {
  float2 h;
  if (F16) h = unpack_f16x2(high);
  else h = make_float2(__uint_as_float(high << 16), __uint_as_float(high & 0xffff0000u));
  return pack2<F16>(a - h.x, b - h.y);
}

// Visible positions of a sequence.
struct Span {
  int lo, hi;      // [lo, hi); hi is the length
  int first, n;    // first tile of 64, number of tiles (one, all hidden, if none is visible)
};
__device__ __forceinline__ Span span_of(const DecodeArgs &a, int b) {
  int len = a.lens[b];
  if (len < 0) len = 0;
  if (len > a.capacity) len = (int)a.capacity;
  int lo = a.starts ? a.starts[b] : 0;
  if (lo < 0) lo = 0;
  if (a.window > 0 && lo < len - a.window) lo = len - a.window;
  Span s{lo, len, lo / kTile, 1};
  if (lo < len) s.n = (len + kTile - 1) / kTile - s.first;
  return s;
}

// A place in the list of all tiles: tile `tile` of group `vh` of sequence b.
struct Cursor {
  int b, vh, tile;
  Span s;
  __device__ __forceinline__ void next(const DecodeArgs &a) {
    if (++tile < s.n) return;
    tile = 0;
    if (++vh < a.n_groups) return;
    vh = 0;
    ++b;
    if (b < a.B) s = span_of(a, b);
  }
};

template <class S>
__global__ void __launch_bounds__(kThreads) decode_kernel(const DecodeArgs a) {
  constexpr int D = S::D, MH = S::MH, NS = S::NS, EV = S::EV;
  constexpr bool Q8 = S::E4M3;
  constexpr int kQRegs = MH == 8 ? 2 : 4;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;  // row and column of the matrix instructions
  float4 *merge = reinterpret_cast<float4 *>(smem + S::kRing);          // [warp][MH][D / 4]
  float2 *ml = reinterpret_cast<float2 *>(smem + S::kRing + S::kMerge);  // [warp][MH]
  int *misc = reinterpret_cast<int *>(smem + S::kRing + S::kMerge + kWarps * MH * 8);

  // ---- this CTA's piece [t0, t1) of the W tiles of all sequences
  int64_t W, t0, t1;
  int n_ctas;
  Cursor cu;
  {
    int64_t *sums = reinterpret_cast<int64_t *>(merge);  // one per warp
    int64_t *place = sums + kWarps;
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      const int len = a.lens[b];
      if (len < 0 || len > a.capacity) set_error(a.err, DEV_ERR_BOUNDS);
      mine += (int64_t)span_of(a, b).n * a.n_groups;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    W = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += sums[w];
      W += sums[w];
    }
    n_ctas = W < (int64_t)gridDim.x ? (int)W : (int)gridDim.x;
    if ((int)blockIdx.x >= n_ctas) return;
    t0 = W * blockIdx.x / n_ctas;
    t1 = W * (blockIdx.x + 1) / n_ctas;
    if (incl - mine <= t0 && t0 < incl) {
      int64_t at = incl - mine;
      int b = b0;
      for (;; ++b) {
        const int64_t n = (int64_t)span_of(a, b).n * a.n_groups;
        if (t0 < at + n) break;
        at += n;
      }
      place[0] = b;
      place[1] = t0 - at;
    }
    __syncthreads();
    cu.b = (int)place[0];
    cu.s = span_of(a, cu.b);
    cu.vh = (int)(place[1] / cu.s.n);
    cu.tile = (int)(place[1] - (int64_t)cu.vh * cu.s.n);
    __syncthreads();  // the merge buffer is free again
  }
  const int n_tiles = (int)(t1 - t0);
  const int G = a.n_heads / a.n_kv;

  // ---- loads: the rows of a warp's 16 keys, a stage ahead of their use
  const uint32_t ring = smem_addr(smem) + warp * (NS * S::kStage);
  Cursor ld = cu;
  int ld_left = n_tiles;
  int32_t page = -1;     // page of this lane's key (lane & 15) of the next tile to load
  int64_t row = 0, srow = 0;
  bool row_on = false;
  auto key_of = [&](const Cursor &k) { return (k.s.first + k.tile) * kTile + warp * kKeys; };
  auto touches = [&](const Cursor &k) {
    const int base = key_of(k);
    return base < k.s.hi && base + kKeys > k.s.lo;
  };
  auto fetch_page = [&]() {
    if (ld_left <= 0) return;
    const int j = key_of(ld) + (lane & 15);
    if (j >= ld.s.lo && j < ld.s.hi)
      page = a.table[ld.b * a.table_stride + (uint32_t)j / (uint32_t)a.kv.page_size];
  };
  auto load_half = [&](int stage, bool is_v) {
    if (ld_left > 0 && touches(ld)) {
      const uint32_t dst = ring + stage * S::kStage + (is_v ? S::kHalfTile : 0);
      if (!is_v) {  // where the lane's key lies; the same for its value row
        const int j = key_of(ld) + (lane & 15);
        row_on = j >= ld.s.lo && j < ld.s.hi;
        if (row_on && (uint64_t)(uint32_t)page >= (uint64_t)a.kv.n_pages) {
          set_error(a.err, DEV_ERR_BOUNDS);
          row_on = false;
        }
        const int slot = (uint32_t)j % (uint32_t)a.kv.page_size;
        const int ch = ld.vh / a.groups_per_kv;
        row = row_on ? page * a.kv.page_stride + ch * a.kv.head_stride + slot * a.kv.slot_stride : 0;
        if (Q8)
          srow = row_on ? page * a.kv.scale_page_stride + ch * a.kv.scale_head_stride +
                              slot * a.kv.scale_slot_stride
                        : 0;
      }
      const uint32_t on = __ballot_sync(0xffffffffu, row_on);
      const uint8_t *base = is_v ? a.kv.v : a.kv.k;
      constexpr int kRowsAtOnce = 32 / S::kPieces;
#pragma unroll
      for (int i = 0; i < kKeys / kRowsAtOnce; ++i) {
        const int r = i * kRowsAtOnce + lane / S::kPieces, p = lane % S::kPieces;
        const int64_t off = __shfl_sync(0xffffffffu, row, r);
        // pieces are exchanged within a row so that the reads below hit all banks
        int q = p;
        if (S::kPieces >= 8) q ^= is_v ? (r & 6) : ((r & 1) << 2);
        else if (is_v) q ^= (r >> 1) & 3;
        copy16(dst + r * S::kRowBytes + q * 16, base + off + p * 16, (on >> r) & 1);
      }
      if (Q8 && !is_v) {  // both scales of a key come with its key row
        const float *from = (lane < kKeys ? a.kv.k_scale : a.kv.v_scale) + srow;
        copy4(ring + stage * S::kStage + 2 * S::kHalfTile + 4 * lane, from, row_on);
      }
    }
    copy_commit();
    if (is_v) {
      if (--ld_left > 0) {
        ld.next(a);
        fetch_page();
      }
    }
  };
  fetch_page();
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    load_half(s, false);
    load_half(s, true);
  }

  // ---- the segment's state
  uint32_t qf[D / 16][kQRegs];
  float o[D / 8][4];
  float m[MH / 8], l[MH / 8], mv[MH / 8];  // mv: the maximum of the weights with value scales
  float qs[MH / 8], sl[MH / 8];            // scale of a raw score, slope * log2(e)
  const float cap2 = a.softcap * kLog2e;
  auto start_segment = [&]() {
    const int ch = cu.vh / a.groups_per_kv, hg = cu.vh - ch * a.groups_per_kv;
    const int in_kv = hg * a.group;
    const int heads = min(a.group, G - in_kv);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
    for (int r = 0; r < MH / 8; ++r) {
      m[r] = mv[r] = -INFINITY;
      l[r] = 0.f;
      const int h = g + 8 * r;
      const bool on = h < heads;
      const int head = ch * G + in_kv + h;
      const __nv_bfloat16 *qp = a.q + (int64_t)cu.b * a.q_stride + (int64_t)head * D;
      uint4 w[D / 32];
#pragma unroll
      for (int s = 0; s < D / 32; ++s) {
        // bf16: piece c + 4s of 8 elements; e4m3: halves of piece c + 4 (s / 2) of 16
        const int at = Q8 ? (c + 4 * (s / 2)) * 16 + 8 * (s & 1) : (c + 4 * s) * 8;
        w[s] = on ? *reinterpret_cast<const uint4 *>(qp + at) : make_uint4(0, 0, 0, 0);
      }
      float unit = a.scale;
      if (!Q8) {
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
          qf[2 * s][r] = w[s].x;
          qf[2 * s + 1][r] = w[s].z;
          qf[2 * s][MH / 8 + r] = w[s].y;
          qf[2 * s + 1][MH / 8 + r] = w[s].w;
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
            const uint32_t f = pack_f16x2(up(__uint_as_float(v << 16)), up(__uint_as_float(v & 0xffff0000u)));
            qf[2 * s + i / 2][(i & 1) * (MH / 8) + r] = f;
          }
      }
      qs[r] = a.softcap > 0.f ? unit / a.softcap : unit * kLog2e;
      sl[r] = a.slopes && on ? a.slopes[head] * kLog2e : 0.f;
    }
  };

  // ---- one tile of 16 keys
  // raw scores, and the scales of this lane's keys (2c and 2c + 1 of both
  // halves of the tile): after this the stage's key rows and scales are free
  auto scores = [&](int stage, float (&s)[2][4], float (&ks)[4], float (&vs)[4]) {
    const uint32_t base = ring + stage * S::kStage;
    if (Q8) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint2 x = lds8(base + 2 * S::kHalfTile + 4 * (8 * t + 2 * c));
        const uint2 y = lds8(base + 2 * S::kHalfTile + 4 * (kKeys + 8 * t + 2 * c));
        ks[2 * t] = __uint_as_float(x.x);
        ks[2 * t + 1] = __uint_as_float(x.y);
        vs[2 * t] = lg2(__uint_as_float(y.x));
        vs[2 * t + 1] = lg2(__uint_as_float(y.y));
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
      const int r = t * 8 + g;
      const uint32_t row_at = base + r * S::kRowBytes;
      const int swz = S::kPieces >= 8 ? (r & 1) << 2 : 0;
      if (!Q8) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 k = lds16(row_at + (((c + 4 * i) ^ swz) << 4));
          const int f = 2 * i;
          mma16816<false>(s[t], qf[f][0], MH == 16 ? qf[f][1] : 0u, qf[f][MH / 8],
                          MH == 16 ? qf[f][kQRegs - 1] : 0u, k.x, k.y);
          mma16816<false>(s[t], qf[f + 1][0], MH == 16 ? qf[f + 1][1] : 0u, qf[f + 1][MH / 8],
                          MH == 16 ? qf[f + 1][kQRegs - 1] : 0u, k.z, k.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint4 k = lds16(row_at + (((c + 4 * i) ^ swz) << 4));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t x = u4_word(k, w);
            const int f = 4 * i + w;
            mma16816<true>(s[t], qf[f][0], MH == 16 ? qf[f][1] : 0u, qf[f][MH / 8],
                           MH == 16 ? qf[f][kQRegs - 1] : 0u, e4m3x2_to_f16x2(x),
                           e4m3x2_to_f16x2(x >> 16));
          }
        }
      }
    }
  };
  // weights of the tile's keys (vs: log2 of their value scales), and the sums
  auto weights = [&](const float (&s)[2][4], const float (&ks)[4], const float (&vs)[4],
                     uint32_t (&p_hi)[MH / 8][2], uint32_t (&p_lo)[MH / 8][2]) {
    const int base = key_of(cu);
    const bool edge = base < cu.s.lo || base + kKeys > cu.s.hi;
#pragma unroll
    for (int r = 0; r < MH / 8; ++r) {
      float x[4], xv[4];
      float top = m[r], top_v = mv[r];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = base + (i >> 1) * 8 + 2 * c + (i & 1);
        float raw = s[i >> 1][2 * r + (i & 1)] * qs[r];
        if (Q8) raw *= ks[i];
        if (a.softcap > 0.f) raw = cap2 * tanh_f32(raw);
        raw = fmaf(sl[r], (float)(key - (cu.s.hi - 1)), raw);
        if (edge && (key < cu.s.lo || key >= cu.s.hi)) raw = -INFINITY;
        x[i] = raw;
        top = fmaxf(top, raw);
        if (Q8) {
          xv[i] = raw == -INFINITY ? -INFINITY : raw + vs[i];
          top_v = fmaxf(top_v, xv[i]);
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float keep = rescale(m[r], top);
      l[r] *= keep;
      float keep_o = keep;
      bool grew = top > m[r];
      m[r] = top;
      if (Q8) {
        top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, 1));
        top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, 2));
        keep_o = rescale(mv[r], top_v);
        grew = top_v > mv[r];
        mv[r] = top_v;
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][2 * r] *= keep_o;
          o[i][2 * r + 1] *= keep_o;
          if (MH == 8) {  // rows 8-15 are the same heads' low parts
            o[i][2] *= keep_o;
            o[i][3] *= keep_o;
          }
        }
      }
      const float zero = top == -INFINITY ? 0.f : top;
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = ex2(x[i] - zero);
        l[r] += p[i];
      }
      if (Q8) {
        const float zero_v = (top_v == -INFINITY ? 0.f : top_v) - kWeightBits;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = ex2(xv[i] - zero_v);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        p_hi[r][t] = pack2<Q8>(p[2 * t], p[2 * t + 1]);
        p_lo[r][t] = pack2_rest<Q8>(p[2 * t], p[2 * t + 1], p_hi[r][t]);
      }
    }
  };
  auto add_values = [&](int stage, const uint32_t (&p_hi)[MH / 8][2], const uint32_t (&p_lo)[MH / 8][2]) {
    const uint32_t vb = ring + stage * S::kStage + S::kHalfTile;
    auto product = [&](float (&acc)[4], uint32_t b0, uint32_t b1) {
      if (MH == 8) {
        mma16816<Q8>(acc, p_hi[0][0], p_lo[0][0], p_hi[0][1], p_lo[0][1], b0, b1);
      } else {
        mma16816<Q8>(acc, p_hi[0][0], p_hi[MH / 8 - 1][0], p_hi[0][1], p_hi[MH / 8 - 1][1], b0, b1);
        if (!Q8)
          mma16816<Q8>(acc, p_lo[0][0], p_lo[MH / 8 - 1][0], p_lo[0][1], p_lo[MH / 8 - 1][1], b0, b1);
      }
    };
#pragma unroll
    for (int h = 0; h < S::H; ++h) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * c + (i & 1) + 8 * (i >> 1);
        const uint32_t row_at = vb + r * S::kRowBytes;
        if (S::kPieces >= 8) {
          v[i] = lds16(row_at + (((g + 8 * h) ^ (r & 6)) << 4));
        } else {  // rows of 64 bytes, half a piece per lane
          const uint2 x = lds8(row_at + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + 8 * (g & 1));
          v[i] = make_uint4(x.x, x.y, 0, 0);
        }
      }
      if (!Q8) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t v0 = u4_word(v[0], w), v1 = u4_word(v[1], w), v2 = u4_word(v[2], w),
                         v3 = u4_word(v[3], w);
          product(o[8 * h + 2 * w], __byte_perm(v0, v1, 0x5410), __byte_perm(v2, v3, 0x5410));
          product(o[8 * h + 2 * w + 1], __byte_perm(v0, v1, 0x7632), __byte_perm(v2, v3, 0x7632));
        }
      } else {
#pragma unroll
        for (int w = 0; w < EV / 4; ++w) {
          const uint32_t v0 = u4_word(v[0], w), v1 = u4_word(v[1], w), v2 = u4_word(v[2], w),
                         v3 = u4_word(v[3], w);
#pragma unroll
          for (int u = 0; u < 2; ++u) {  // codes 2u, 2u + 1 of the word, keys paired
            const uint32_t x = __byte_perm(v0, v1, u ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(v2, v3, u ? 0x7362 : 0x5140);
            product(o[EV * h + 4 * w + 2 * u], e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y));
            product(o[EV * h + 4 * w + 2 * u + 1], e4m3x2_to_f16x2(x >> 16), e4m3x2_to_f16x2(y >> 16));
          }
        }
      }
    }
  };

  // ---- end of a segment, or of this CTA's piece of it
  // Outputs are kept as float4 items: item i of a head is elements d(i) .. d(i) + 3.
  auto element_of = [&](int i) {
    const int cc = i & 3, q = i >> 2, jj = q % (EV / 4), hu = q / (EV / 4);
    return (2 * cc + (hu & 1) + 8 * (hu >> 1)) * EV + 4 * jj;
  };
  auto write_out = [&](int b, int head, int item, float4 v, float mm, float ll) {
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const int64_t bh = (int64_t)b * a.n_heads + head;
    uint2 w;
    w.x = pack2<false>(v.x * inv, v.y * inv);
    w.y = pack2<false>(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2 *>(a.out + bh * D + element_of(item)) = w;
    if (item == 0 && a.lse) a.lse[bh] = (mm + log2f(ll)) * kLn2;
  };
  auto finish_segment = [&](int64_t seg0, int64_t seg1) {
    const int ch = cu.vh / a.groups_per_kv, hg = cu.vh - ch * a.groups_per_kv;
    const int in_kv = hg * a.group, heads = min(a.group, G - in_kv);
    const int head0 = ch * G + in_kv;
#pragma unroll
    for (int r = 0; r < MH / 8; ++r) {
      float sum = l[r];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      float f = 1.f;
      if (Q8 && m[r] != -INFINITY && mv[r] != -INFINITY) f = ex2(mv[r] - m[r] - kWeightBits);
      const int h = g + 8 * r;
      float4 *dst = merge + (warp * MH + h) * (D / 4);
#pragma unroll
      for (int hh = 0; hh < S::H; ++hh)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int jj = 0; jj < EV / 4; ++jj) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float *x = o[EV * hh + 4 * jj + i];
              v[i] = (MH == 8 ? x[u] + x[2 + u] : x[2 * r + u]) * f;
            }
            dst[((hh * 2 + u) * (EV / 4) + jj) * 4 + c] = make_float4(v[0], v[1], v[2], v[3]);
          }
      if (c == 0) ml[warp * MH + h] = make_float2(m[r], sum);
    }
    __syncthreads();
    // which CTAs hold pieces of this segment
    int first = blockIdx.x, pieces = 1;
    if (seg0 < t0 || seg1 > t1) {
      first = (int)(((seg0 + 1) * n_ctas - 1) / W);
      pieces = (int)((seg1 * n_ctas - 1) / W) - first + 1;
    }
    const int items = heads * (D / 4);
    float4 *part = reinterpret_cast<float4 *>(a.part);
    float2 *part_ml = reinterpret_cast<float2 *>(a.part_ml);
    // a CTA's own slots: 0 for a segment that began before its piece, 1 otherwise
    auto slot_of = [&](int piece) { return 2 * (first + piece) + (piece == 0 ? 1 : 0); };
    const int mine = slot_of(blockIdx.x - first);
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
        const float4 x = merge[(w * MH + h) * (D / 4) + it];
        ll = fmaf(f, s.y, ll);
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
      }
      if (pieces == 1) {
        write_out(cu.b, head0 + h, it, v, mm, ll);
      } else {
        part[((int64_t)mine * a.group + h) * (D / 4) + it] = v;
        if (it == 0) part_ml[(int64_t)mine * a.group + h] = make_float2(mm, ll);
      }
    }
    if (pieces > 1) {
      // joins `n` pieces, every `step`-th from piece p0 on; true where this CTA arrived last
      auto arrive = [&](int *counter, int n) {
        __syncthreads();
        if (threadIdx.x == 0) {
          __threadfence();
          const int before = atomicAdd(counter, 1);
          const bool last = before == n - 1;
          if (last) *counter = 0;  // for the next call
          __threadfence();
          misc[0] = last;
        }
        __syncthreads();
        return misc[0] != 0;
      };
      auto join = [&](int p0, int step, int n, bool final) {
        for (int i = threadIdx.x; i < items; i += kThreads) {
          const int h = i / (D / 4), it = i % (D / 4);
          float mm = -INFINITY, ll = 0.f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p = 0; p < n; p += 4) {
            float2 s[4];
            float4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const bool on = p + k < n;
              const int64_t at = (int64_t)slot_of(p0 + (on ? p + k : 0) * step) * a.group + h;
              s[k] = __ldcg(part_ml + at);
              x[k] = __ldcg(part + at * (D / 4) + it);
              if (!on) {
                s[k] = make_float2(-INFINITY, 0.f);
                x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              }
            }
            float top = mm;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, s[k].x);
            const float f0 = rescale(mm, top);
            ll *= f0;
            v.x *= f0;
            v.y *= f0;
            v.z *= f0;
            v.w *= f0;
            mm = top;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float f = rescale(s[k].x, top);
              ll = fmaf(f, s[k].y, ll);
              v.x = fmaf(f, x[k].x, v.x);
              v.y = fmaf(f, x[k].y, v.y);
              v.z = fmaf(f, x[k].z, v.z);
              v.w = fmaf(f, x[k].w, v.w);
            }
          }
          if (final) {
            write_out(cu.b, head0 + h, it, v, mm, ll);
          } else {  // in place of the group's first piece, which only this thread has read ..
            part[((int64_t)slot_of(p0) * a.group + h) * (D / 4) + it] = v;
            if (it == 0) ml[h] = make_float2(mm, ll);  // .. except for its statistics
          }
        }
        if (!final) {
          __syncthreads();
          for (int h = threadIdx.x; h < heads; h += kThreads)
            part_ml[(int64_t)slot_of(p0) * a.group + h] = ml[h];
        }
      };
      // Counters: a CTA is the first of at most one shared segment and a later
      // piece's holder of at most one other, so three arrays by CTA do.
      const int piece = blockIdx.x - first, grp = piece / kJoin;
      const int p0 = grp * kJoin, in_grp = min(kJoin, pieces - p0);
      const int groups = (pieces + kJoin - 1) / kJoin;
      if (arrive(a.counters + (grp == 0 ? 0 : a.max_ctas) + first + p0, in_grp)) {
        join(p0, 1, in_grp, groups == 1);
        if (groups > 1 && arrive(a.counters + 2 * a.max_ctas + first, groups))
          join(0, kJoin, groups, true);
      }
    }
    __syncthreads();  // the merge buffer is free again
  };

  int stage = 0;
  for (int i = 0; i < n_tiles; ++i) {
    if (i == 0 || cu.tile == 0) start_segment();
    const bool on = touches(cu);
    uint32_t p_hi[MH / 8][2], p_lo[MH / 8][2];
    float s[2][4], ks[4], vs[4];
    copy_wait<2 * NS - 1>();  // the key rows
    __syncwarp();
    if (on) scores(stage, s, ks, vs);
    __syncwarp();
    load_half(stage, false);
    if (on) weights(s, ks, vs, p_hi, p_lo);
    copy_wait<2 * NS - 1>();  // the value rows
    __syncwarp();
    if (on) add_values(stage, p_hi, p_lo);
    __syncwarp();
    load_half(stage, true);
    if (cu.tile == cu.s.n - 1 || i == n_tiles - 1)
      finish_segment(t0 + i - cu.tile, t0 + i - cu.tile + cu.s.n);
    if (i + 1 < n_tiles) cu.next(a);
    stage = stage + 1 == NS ? 0 : stage + 1;
  }
  copy_wait<0>();
}

template <class S>
cudaError_t launch_shape(const DecodeArgs &a, int grid, cudaStream_t s) {
  decode_kernel<S><<<grid, kThreads, S::kSmem, s>>>(a);
  return cudaGetLastError();
}
template <class S>
cudaError_t plan_shape(int *ctas_per_sm) {
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas_per_sm, decode_kernel<S>, kThreads, S::kSmem);
}

// Calls f with the shape of (d, e4m3, heads of a group).
template <class F>
cudaError_t with_shape(int d, bool e4m3, int group, F f) {
  const bool wide = group > 8;
  switch (d) {
    case 64:
      if (e4m3) return wide ? f(Shape<64, true, 16, 4>{}) : f(Shape<64, true, 8, 4>{});
      return wide ? f(Shape<64, false, 16, 3>{}) : f(Shape<64, false, 8, 3>{});
    case 128:
      if (e4m3) return wide ? f(Shape<128, true, 16, 3>{}) : f(Shape<128, true, 8, 3>{});
      return wide ? f(Shape<128, false, 16, 2>{}) : f(Shape<128, false, 8, 2>{});
    case 256:
      if (e4m3) return wide ? f(Shape<256, true, 16, 2>{}) : f(Shape<256, true, 8, 2>{});
      return wide ? f(Shape<256, false, 16, 1>{}) : f(Shape<256, false, 8, 1>{});
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int decode_group(int heads_per_kv) {
  const int n = (heads_per_kv + 15) / 16;
  return (heads_per_kv + n - 1) / n;
}

int64_t decode_tiles(int64_t positions) { return (positions + kTile - 1) / kTile; }

cudaError_t plan_paged_decode(int d, bool e4m3, int group, int *ctas_per_sm) {
  return with_shape(d, e4m3, group, [&](auto s) { return plan_shape<decltype(s)>(ctas_per_sm); });
}

cudaError_t launch_paged_decode(const DecodeArgs &a, int d, bool e4m3, int grid, cudaStream_t s) {
  return with_shape(d, e4m3, a.group, [&](auto sh) { return launch_shape<decltype(sh)>(a, grid, s); });
}

}  // namespace fp8moe
