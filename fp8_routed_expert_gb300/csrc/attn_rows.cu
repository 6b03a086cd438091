// Head rows on their way into and out of the paged key/value cache: norm and
// rotation of query and key heads in one pass, quantisation as a row is
// written, and the rows read back (moe_attn_norm_rope, _append, _write,
// _read).
//
// A head row of d elements is held by d / 8 neighbouring lanes, 8 elements (16
// bytes) each.  The sum of squares and the largest magnitude of a row are
// shuffles within its lanes.  In the half-split rotation the partner of an
// element is R/2 away, R/16 lanes further on, and comes by a shuffle too;
// interleaved pairs lie within a lane.
//
// Angles.  position * freq / 2 pi is only needed modulo 1.  With the frequency
// as a 64-bit fraction of a turn, the 64-bit integer product wraps exactly
// modulo one turn: the error is 2^-65 turns times the position (2^-34 at the
// end of the int32 range) where an f32 product would lose the angle of a far
// position altogether.
#include "common.cuh"
#include "paged_attn.h"

namespace fp8moe {

namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = u4_word(v, i);
    f[2 * i] = __uint_as_float(w << 16);
    f[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Sum / maximum over the L neighbouring lanes of a row (L a power of two).
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Smallest e >= -126 with amax <= 448 * 2^e; 0 for an all-zero row.  amax is
// finite.  448 = 0.875 * 2^9, so with amax = m * 2^x, m in [0.5, 1), e is x - 9,
// or one more when m > 0.875; no division, no rounding.
__device__ __forceinline__ int e4m3_row_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  int x;
  const float m = frexpf(amax, &x);
  const int e = x - 9 + (m > 0.875f ? 1 : 0);
  return e < -126 ? -126 : e;
}

// Where a token's rows go: byte offset of its row in key/value head 0, offset
// of that row's scale; row < 0 for nowhere.
struct Place {
  int64_t row, scale;
};
__device__ __forceinline__ Place place_of(int64_t slot, const KvView &kv, int *err) {
  if (slot < 0) return Place{-1, 0};
  int64_t page;
  int at;
  if (slot <= 0x7fffffff) {  // the usual case, without a 64-bit division
    const uint32_t q = (uint32_t)slot / (uint32_t)kv.page_size;
    page = q;
    at = (int)((uint32_t)slot - q * (uint32_t)kv.page_size);
  } else {
    page = slot / kv.page_size;
    at = (int)(slot - page * kv.page_size);
  }
  if (page >= kv.n_pages) {
    set_error(err, DEV_ERR_BOUNDS);
    return Place{-1, 0};
  }
  return Place{page * kv.page_stride + at * kv.slot_stride,
               page * kv.scale_page_stride + at * kv.scale_slot_stride};
}

// How a launch cuts T tokens of n_rows rows each over CTAs that take at most
// kDepth rows per group of lanes: `tokens` whole tokens per CTA, or (tokens ==
// 1) `rows` rows of one token, the others in further CTAs along y.
constexpr int kDepth = 4;       // rows of a lane group, all loaded before the first is used
constexpr int kMaxTokens = 8;
struct RowCut {
  int tokens, rows;
  uint32_t mul;  // item / n_rows = item * mul >> 20 for items of several tokens
};
template <int D>
RowCut cut_rows(int64_t T, int n_rows, int sms) {
  constexpr int kRows = kRowThreads / (D / 8);
  const int64_t want = 2 * (int64_t)sms;  // CTAs that keep every SM busy
  RowCut c{1, kRows, 0};
  int depth = kDepth;
  while (depth > 1 && T * ((n_rows + depth * kRows - 1) / (depth * kRows)) < want) depth /= 2;
  c.rows = depth * kRows;
  if (n_rows <= c.rows) {
    c.rows = n_rows;
    int64_t n = kDepth * kRows / n_rows;
    if (n > kMaxTokens) n = kMaxTokens;
    if (n > T / want) n = T / want;
    if (n > 1) {
      c.tokens = (int)n;
      c.mul = ((1u << 20) + n_rows - 1) / n_rows;  // exact while items * n_rows < 2^20
    }
  }
  return c;
}

// Grid (token groups, row blocks); items of a CTA: (token, row).  Bound by HBM:
// every row is read and written once, a lane's rows are all in flight before
// the angles are computed, and the angles of a token are computed once for all
// its heads.
template <int D>
__global__ void __launch_bounds__(kRowThreads) head_rows_kernel(const __grid_constant__ RowArgs a,
                                                                const RowCut cut) {
  constexpr int L = D / 8, kRows = kRowThreads / L;
  // cos and sin of the tokens' angles, pieces of four swapped so that lanes 32
  // bytes apart use all banks
  __shared__ __align__(16) float cs[kMaxTokens][2][D / 2];
  __shared__ Place at[kMaxTokens];
  const int lane = threadIdx.x % L, slot0 = threadIdx.x / L;
  const int n_rows = a.n_q + a.n_k + a.n_v;
  const int64_t t_base = (int64_t)blockIdx.x * cut.tokens;
  const int tokens = (int)min((int64_t)cut.tokens, a.T - t_base);
  const int r_base = blockIdx.y * cut.rows;
  const int items = cut.tokens > 1 ? tokens * n_rows : min(cut.rows, n_rows - r_base);
  const auto token_of = [&](int i) { return cut.tokens > 1 ? (int)((i * cut.mul) >> 20) : 0; };
  uint4 raw[kDepth];
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    const int i = slot0 + k * kRows;
    raw[k] = make_uint4(0, 0, 0, 0);
    if (i < items) {
      const int tl = token_of(i), r = r_base + i - tl * n_rows;
      const bool is_q = r < a.n_q, is_k = !is_q && r < a.n_q + a.n_k;
      const int h = is_q ? r : (is_k ? r - a.n_q : r - a.n_q - a.n_k);
      const RowsIn &in = is_q ? a.q : (is_k ? a.k : a.v);
      raw[k] = *reinterpret_cast<const uint4 *>(in.p + (t_base + tl) * in.stride + h * D + lane * 8);
    }
  }
  if (a.half > 0) {
    for (int i = threadIdx.x; i < tokens * a.half; i += kRowThreads) {
      const int tl = i / a.half, f = i - tl * a.half;
      const uint64_t pos = (uint64_t)(int64_t)a.positions[t_base + tl];
      // signed fraction of a turn in [-1/2, 1/2), as half turns for sincospi
      const float x = (float)(int64_t)(pos * a.turns[f]) * 0x1p-63f;
      float sn, cn;
      sincospif(x, &sn, &cn);
      const int piece = f / 4, place = (piece ^ ((piece >> 3) & 1)) * 4 + f % 4;
      cs[tl][0][place] = cn;
      cs[tl][1][place] = sn;
    }
  }
  if (a.cache && threadIdx.x < tokens) at[threadIdx.x] = place_of(a.slots[t_base + threadIdx.x], a.kv, a.err);
  __syncthreads();
  const int step = a.half / 8;  // lanes between the two halves of a rotated row
  const bool second = lane >= step;
  const int partner = (second ? lane - step : lane + step) & (L - 1);
  const auto angles = [&](int tl, int which, int piece) {
    return *reinterpret_cast<const float4 *>(&cs[tl][which][(piece ^ ((piece >> 3) & 1)) * 4]);
  };
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    if (k * kRows >= items) break;  // the same for the whole CTA: shuffles take whole warps
    const int i = slot0 + k * kRows;
    const bool on = i < items;
    const int tl = on ? token_of(i) : 0, r = r_base + i - tl * n_rows;
    const int64_t t = t_base + tl;
    const bool is_q = r < a.n_q, is_k = !is_q && r < a.n_q + a.n_k;
    const int h = is_q ? r : (is_k ? r - a.n_q : r - a.n_q - a.n_k);
    float y[8];
    unpack8(raw[k], y);
    if (a.q_weight != nullptr || a.k_weight != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
      ss = row_sum<L>(ss);
      const float *w = is_q ? a.q_weight : (is_k ? a.k_weight : nullptr);
      if (w != nullptr) {
        const float rms = __frsqrt_rn(fmaf(ss, 1.0f / D, a.eps));
        const float4 w0 = __ldg(reinterpret_cast<const float4 *>(w) + 2 * lane);
        const float4 w1 = __ldg(reinterpret_cast<const float4 *>(w) + 2 * lane + 1);
        y[0] = y[0] * rms * w0.x;
        y[1] = y[1] * rms * w0.y;
        y[2] = y[2] * rms * w0.z;
        y[3] = y[3] * rms * w0.w;
        y[4] = y[4] * rms * w1.x;
        y[5] = y[5] * rms * w1.y;
        y[6] = y[6] * rms * w1.z;
        y[7] = y[7] * rms * w1.w;
      }
    }
    if (a.half > 0) {
      const bool turned = (is_q || is_k) && lane * 8 < 2 * a.half;
      if (a.interleaved) {
        if (turned) {
          const float4 cn = angles(tl, 0, lane), sn = angles(tl, 1, lane);
          const float cc[4] = {cn.x, cn.y, cn.z, cn.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float u = y[2 * j], v = y[2 * j + 1];
            y[2 * j] = u * cc[j] - v * ss[j];
            y[2 * j + 1] = v * cc[j] + u * ss[j];
          }
        }
      } else {
        float z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = __shfl_sync(0xffffffffu, y[j], partner, L);
        if (turned) {
          const int p = 2 * (second ? lane - step : lane);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 cn = angles(tl, 0, p + q), sn = angles(tl, 1, p + q);
            const float cc[4] = {cn.x, cn.y, cn.z, cn.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float s1 = second ? ss[j] : -ss[j];
              y[4 * q + j] = fmaf(z[4 * q + j], s1, y[4 * q + j] * cc[j]);
            }
          }
        }
      }
    }
    if (is_q || !a.cache) {
      if (on) {
        const RowsOut &out = is_q ? a.q_out : a.k_out;
        *reinterpret_cast<uint4 *>(out.p + t * out.stride + h * D + lane * 8) = pack8(y);
      }
      if (!a.cache || !a.e4m3) continue;
    }
    const Place place = at[tl];
    const bool store = on && !is_q && place.row >= 0;
    uint8_t *row = (is_k ? a.kv.k : a.kv.v) + (store ? place.row + h * a.kv.head_stride : 0);
    if (!a.e4m3) {
      if (store) *reinterpret_cast<uint4 *>(row + lane * 16) = pack8(y);
      continue;
    }
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float m = fabsf(y[j]);
      if (m < INFINITY) amax = fmaxf(amax, m);
      else y[j] = NAN;  // an infinity has no code; a NaN stays one
    }
    amax = row_max<L>(amax);
    if (store) {
      const int e = e4m3_row_exponent(amax);  // in [-126, 120]
      const float down = exp2i(-e);
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[j] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * j] * down, y[2 * j + 1] * down),
                                        __NV_SATFINITE, __NV_E4M3);
      *reinterpret_cast<uint2 *>(row + lane * 8) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      if (lane == 0)
        (is_k ? a.kv.k_scale : a.kv.v_scale)[place.scale + h * a.kv.scale_head_stride] = exp2i(e);
    }
  }
}

// Rows out of the cache, cut over CTAs like the rows in.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) read_rows_kernel(const __grid_constant__ ReadArgs a,
                                                                const RowCut cut) {
  constexpr int L = D / 8, kRows = kRowThreads / L;
  __shared__ Place at[kMaxTokens];
  const int lane = threadIdx.x % L, slot0 = threadIdx.x / L;
  const int n_rows = 2 * a.n_kv;
  const int64_t t_base = (int64_t)blockIdx.x * cut.tokens;
  const int tokens = (int)min((int64_t)cut.tokens, a.T - t_base);
  const int r_base = blockIdx.y * cut.rows;
  const int items = cut.tokens > 1 ? tokens * n_rows : min(cut.rows, n_rows - r_base);
  const auto token_of = [&](int i) { return cut.tokens > 1 ? (int)((i * cut.mul) >> 20) : 0; };
  if (threadIdx.x < tokens) at[threadIdx.x] = place_of(a.slots[t_base + threadIdx.x], a.kv, a.err);
  __syncthreads();
  uint4 raw[kDepth];
  float scale[kDepth];
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    const int i = slot0 + k * kRows;
    raw[k] = make_uint4(0, 0, 0, 0);
    scale[k] = 0.f;
    if (i < items) {
      const int tl = token_of(i), r = r_base + i - tl * n_rows;
      const bool is_k = r < a.n_kv;
      const int h = is_k ? r : r - a.n_kv;
      const Place place = at[tl];
      if (place.row >= 0) {
        const uint8_t *row = (is_k ? a.kv.k : a.kv.v) + place.row + h * a.kv.head_stride;
        if (E4M3) {
          const uint2 c = *reinterpret_cast<const uint2 *>(row + lane * 8);
          raw[k].x = c.x;
          raw[k].y = c.y;
          scale[k] = (is_k ? a.kv.k_scale : a.kv.v_scale)[place.scale + h * a.kv.scale_head_stride];
        } else {
          raw[k] = *reinterpret_cast<const uint4 *>(row + lane * 16);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    const int i = slot0 + k * kRows;
    if (i >= items) break;
    const int tl = token_of(i), r = r_base + i - tl * n_rows;
    const bool is_k = r < a.n_kv;
    const int h = is_k ? r : r - a.n_kv;
    if (E4M3) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = unpack_f16x2(e4m3x2_to_f16x2((j < 2 ? raw[k].x : raw[k].y) >> (16 * (j & 1))));
        f[2 * j] = v.x * scale[k];
        f[2 * j + 1] = v.y * scale[k];
      }
      raw[k] = pack8(f);
    }
    const RowsOut &out = is_k ? a.k_out : a.v_out;
    *reinterpret_cast<uint4 *>(out.p + (t_base + tl) * out.stride + h * D + lane * 8) = raw[k];
  }
}

dim3 grid_of(const RowCut &c, int64_t T, int n_rows) {
  return dim3((unsigned)((T + c.tokens - 1) / c.tokens),
              c.tokens > 1 ? 1u : (unsigned)((n_rows + c.rows - 1) / c.rows));
}

template <int D>
cudaError_t rows_of(const RowArgs &a, cudaStream_t s) {
  const int n_rows = a.n_q + a.n_k + a.n_v;
  const RowCut c = cut_rows<D>(a.T, n_rows, a.sms);
  head_rows_kernel<D><<<grid_of(c, a.T, n_rows), kRowThreads, 0, s>>>(a, c);
  return cudaGetLastError();
}

template <int D>
cudaError_t read_of(const ReadArgs &a, cudaStream_t s) {
  const RowCut c = cut_rows<D>(a.T, 2 * a.n_kv, a.sms);
  const dim3 grid = grid_of(c, a.T, 2 * a.n_kv);
  if (a.e4m3) read_rows_kernel<D, true><<<grid, kRowThreads, 0, s>>>(a, c);
  else read_rows_kernel<D, false><<<grid, kRowThreads, 0, s>>>(a, c);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows(const RowArgs &a, int d, cudaStream_t s) {
  switch (d) {
    case 64: return rows_of<64>(a, s);
    case 128: return rows_of<128>(a, s);
    case 256: return rows_of<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_read(const ReadArgs &a, int d, cudaStream_t s) {
  switch (d) {
    case 64: return read_of<64>(a, s);
    case 128: return read_of<128>(a, s);
    case 256: return read_of<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fp8moe
