// Head rows on their way into and out of the paged key/value cache: norm and
// rotation of query and key heads in one pass, quantisation as a row is
// written, and the rows read back (moe_attn_norm_rope, _append, _write,
// _read).
//
// A head row of d elements is held by d / 16 neighbouring lanes, 16 elements in
// two pieces of 8 (16 bytes) each.  Lane i of a rotated row takes the pieces at
// 8i and R/2 + 8i in the half-split rotation, those at 16i and 16i + 8 in the
// interleaved one: either way both elements of a pair are its own and its angles
// are 8i .. 8i + 7.  The remaining pieces go to the remaining lanes in order.
// Only the sum of squares and the largest magnitude of a row cross lanes.
//
// Angles.  position * freq / 2 pi is only needed modulo 1.  With the frequency
// as a 64-bit fraction of a turn, the 64-bit integer product wraps exactly
// modulo one turn: the error is 2^-65 turns times the position (2^-34 at the
// end of the int32 range) where an f32 product would lose the angle of a far
// position altogether.
#include "common.cuh"
#include "kernels.h"
#include "paged_attn.h"

namespace fp8moe {

namespace {

constexpr int kRowThreads = 128;

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
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
constexpr int kDepth = 2;  // rows of a lane group, all loaded before the first is used
constexpr int kMaxTokens = 8;
struct RowCut {
  int tokens, rows;
  uint32_t mul;  // item / n_rows = item * mul >> 20 for items of several tokens
};
template <int D>
RowCut cut_rows(int64_t T, int n_rows, int sms) {
  constexpr int kRows = kRowThreads / (D / 16);
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

__device__ __forceinline__ uint2 e4m3x8(const float (&y)[16], int from, float scale) {
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    c[j] = __nv_cvt_float2_to_fp8x2(make_float2(y[from + 2 * j] * scale, y[from + 2 * j + 1] * scale),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Grid (token groups, row blocks); items of a CTA: (token, row).  Every row is
// read and written once; a lane's rows are all in flight before the angles are
// computed, and the angles of a token are computed once for all its heads.
// Issue slots bound it next to HBM, hence the layout above without shuffles of
// the row itself.
template <int D>
__global__ void __launch_bounds__(kRowThreads) head_rows_kernel(const __grid_constant__ RowArgs a,
                                                                const RowCut cut) {
  constexpr int L = D / 16, kRows = kRowThreads / L;
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
  // this lane's pieces
  const bool turned = lane * 8 < a.half;
  const int o0 = turned && !a.interleaved ? 8 * lane : 16 * lane;
  const int o1 = turned && !a.interleaved ? a.half + 8 * lane : 16 * lane + 8;
  struct Item {
    int tl, h;
    bool on, is_q, is_k;
  };
  const auto item = [&](int k) {
    Item it;
    const int i = slot0 + k * kRows;
    it.on = i < items;
    it.tl = cut.tokens > 1 && it.on ? (int)((i * cut.mul) >> 20) : 0;
    const int r = r_base + i - it.tl * n_rows;
    it.is_q = r < a.n_q;
    it.is_k = !it.is_q && r < a.n_q + a.n_k;
    it.h = r - (it.is_q ? 0 : (it.is_k ? a.n_q : a.n_q + a.n_k));
    return it;
  };
  pdl_wait();
  pdl_trigger();
  uint4 raw[kDepth][2];
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    const Item it = item(k);
    raw[k][0] = raw[k][1] = make_uint4(0, 0, 0, 0);
    if (it.on) {
      const __nv_bfloat16 *p = it.is_q ? a.q.p : (it.is_k ? a.k.p : a.v.p);
      const int64_t stride = it.is_q ? a.q.stride : (it.is_k ? a.k.stride : a.v.stride);
      p += (t_base + it.tl) * stride + it.h * D;
      raw[k][0] = *reinterpret_cast<const uint4 *>(p + o0);
      raw[k][1] = *reinterpret_cast<const uint4 *>(p + o1);
    }
  }
  if (a.half > 0) {
    for (int i = threadIdx.x; i < tokens * a.half; i += kRowThreads) {
      const int tl = cut.tokens > 1 ? i / a.half : 0, f = i - tl * a.half;
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
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    if (k * kRows >= items) break;  // the same for the whole CTA: shuffles take whole warps
    const Item it = item(k);
    float y[16];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = u4_word(raw[k][p], j);
        y[8 * p + 2 * j] = __uint_as_float(w << 16);
        y[8 * p + 2 * j + 1] = __uint_as_float(w & 0xffff0000u);
      }
    if (a.q_weight != nullptr || a.k_weight != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) ss = fmaf(y[j], y[j], ss);
      ss = row_sum<L>(ss);
      const float *w = it.is_q ? a.q_weight : (it.is_k ? a.k_weight : nullptr);
      if (w != nullptr) {
        const float rms = __frsqrt_rn(fmaf(ss, 1.0f / D, a.eps));
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float4 v = __ldg(reinterpret_cast<const float4 *>(w + (p < 2 ? o0 : o1)) + (p & 1));
          y[4 * p] = y[4 * p] * rms * v.x;
          y[4 * p + 1] = y[4 * p + 1] * rms * v.y;
          y[4 * p + 2] = y[4 * p + 2] * rms * v.z;
          y[4 * p + 3] = y[4 * p + 3] * rms * v.w;
        }
      }
    }
    if (turned && (it.is_q || it.is_k)) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int piece = 2 * lane + q, place = (piece ^ ((piece >> 3) & 1)) * 4;
        const float4 c4 = *reinterpret_cast<const float4 *>(&cs[it.tl][0][place]);
        const float4 s4 = *reinterpret_cast<const float4 *>(&cs[it.tl][1][place]);
        const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float &u = y[8 * q + 2 * j], &v = y[8 * q + 2 * j + 1];
            const float u0 = u;
            u = fmaf(-v, ss[j], u * cc[j]);
            v = fmaf(u0, ss[j], v * cc[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float &u = y[4 * q + j], &v = y[8 + 4 * q + j];
            const float u0 = u;
            u = fmaf(-v, ss[j], u * cc[j]);
            v = fmaf(u0, ss[j], v * cc[j]);
          }
        }
      }
    }
    const bool to_cache = a.cache && !it.is_q;
    if (it.on && (!to_cache || !a.e4m3)) {
      uint4 w[2];
#pragma unroll
      for (int p = 0; p < 2; ++p)
        w[p] = make_uint4(pack_bf16x2(y[8 * p], y[8 * p + 1]), pack_bf16x2(y[8 * p + 2], y[8 * p + 3]),
                          pack_bf16x2(y[8 * p + 4], y[8 * p + 5]), pack_bf16x2(y[8 * p + 6], y[8 * p + 7]));
      __nv_bfloat16 *out;
      if (to_cache) {
        out = reinterpret_cast<__nv_bfloat16 *>((it.is_k ? a.kv.k : a.kv.v) + at[it.tl].row +
                                                it.h * a.kv.head_stride);
      } else {
        out = it.is_q ? a.q_out.p : a.k_out.p;
        out += (t_base + it.tl) * (it.is_q ? a.q_out.stride : a.k_out.stride) + it.h * D;
      }
      if (!to_cache || at[it.tl].row >= 0) {
        *reinterpret_cast<uint4 *>(out + o0) = w[0];
        *reinterpret_cast<uint4 *>(out + o1) = w[1];
      }
    }
    if (!a.e4m3) continue;
    float amax = 0.f;  // fmaxf passes over a NaN, which stays one in its code
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(y[j]));
    amax = row_max<L>(amax);
    if (__any_sync(0xffffffffu, amax == INFINITY)) {  // an infinity has no code: it becomes a NaN
      float fin = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (fabsf(y[j]) == INFINITY) y[j] = NAN;
        fin = fmaxf(fin, fabsf(y[j]));
      }
      amax = row_max<L>(fin);
    }
    const Place place = at[it.tl];
    if (it.on && to_cache && place.row >= 0) {
      const int e = e4m3_row_exponent(amax);  // in [-126, 120]
      const float down = exp2i(-e);
      uint8_t *row = (it.is_k ? a.kv.k : a.kv.v) + place.row + it.h * a.kv.head_stride;
      *reinterpret_cast<uint2 *>(row + o0) = e4m3x8(y, 0, down);
      *reinterpret_cast<uint2 *>(row + o1) = e4m3x8(y, 8, down);
      if (lane == 0)
        (it.is_k ? a.kv.k_scale : a.kv.v_scale)[place.scale + it.h * a.kv.scale_head_stride] = exp2i(e);
    }
  }
}

// Rows out of the cache, cut over CTAs like the rows in: a lane takes 16
// consecutive elements.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) read_rows_kernel(const __grid_constant__ ReadArgs a,
                                                                const RowCut cut) {
  constexpr int L = D / 16, kRows = kRowThreads / L;
  __shared__ Place at[kMaxTokens];
  const int lane = threadIdx.x % L, slot0 = threadIdx.x / L;
  const int n_rows = 2 * a.n_kv;
  const int64_t t_base = (int64_t)blockIdx.x * cut.tokens;
  const int tokens = (int)min((int64_t)cut.tokens, a.T - t_base);
  const int r_base = blockIdx.y * cut.rows;
  const int items = cut.tokens > 1 ? tokens * n_rows : min(cut.rows, n_rows - r_base);
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < tokens) at[threadIdx.x] = place_of(a.slots[t_base + threadIdx.x], a.kv, a.err);
  __syncthreads();
  uint4 raw[kDepth][2];
  float scale[kDepth];
  __nv_bfloat16 *out[kDepth];
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    const int i = slot0 + k * kRows;
    raw[k][0] = raw[k][1] = make_uint4(0, 0, 0, 0);
    scale[k] = 0.f;
    out[k] = nullptr;
    if (i < items) {
      const int tl = cut.tokens > 1 ? (int)((i * cut.mul) >> 20) : 0, r = r_base + i - tl * n_rows;
      const bool is_k = r < a.n_kv;
      const int h = is_k ? r : r - a.n_kv;
      out[k] = (is_k ? a.k_out.p : a.v_out.p) + (t_base + tl) * (is_k ? a.k_out.stride : a.v_out.stride) +
               h * D + 16 * lane;
      const Place place = at[tl];
      if (place.row >= 0) {
        const uint4 *row = reinterpret_cast<const uint4 *>((is_k ? a.kv.k : a.kv.v) + place.row +
                                                           h * a.kv.head_stride);
        if (E4M3) {
          raw[k][0] = row[lane];
          scale[k] = (is_k ? a.kv.k_scale : a.kv.v_scale)[place.scale + h * a.kv.scale_head_stride];
        } else {
          raw[k][0] = row[2 * lane];
          raw[k][1] = row[2 * lane + 1];
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    if (out[k] == nullptr) break;
    if (E4M3) {
      const uint4 c = raw[k][0];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = u4_word(c, 2 * p + j / 2) >> (16 * (j & 1));
          const float2 v = unpack_f16x2(e4m3x2_to_f16x2(x));
          w[j] = pack_bf16x2(v.x * scale[k], v.y * scale[k]);
        }
        raw[k][p] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    reinterpret_cast<uint4 *>(out[k])[0] = raw[k][0];
    reinterpret_cast<uint4 *>(out[k])[1] = raw[k][1];
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
  return launch_pdl(head_rows_kernel<D>, grid_of(c, a.T, n_rows), dim3(kRowThreads), 0, s, a, c);
}

template <int D>
cudaError_t read_of(const ReadArgs &a, cudaStream_t s) {
  const RowCut c = cut_rows<D>(a.T, 2 * a.n_kv, a.sms);
  const dim3 grid = grid_of(c, a.T, 2 * a.n_kv);
  return launch_pdl(a.e4m3 ? read_rows_kernel<D, true> : read_rows_kernel<D, false>, grid,
                    dim3(kRowThreads), 0, s, a, c);
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
