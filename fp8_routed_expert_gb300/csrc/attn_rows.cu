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

// Where a token's rows go: page and slot within it, or page -1 for nowhere.
struct Place {
  int64_t page;
  int slot;
};
__device__ __forceinline__ Place place_of(int64_t slot, const KvView &kv, int *err) {
  if (slot < 0) return Place{-1, 0};
  Place p;
  if (slot <= 0x7fffffff) {  // the usual case, without a 64-bit division
    const uint32_t q = (uint32_t)slot / (uint32_t)kv.page_size;
    p = Place{(int64_t)q, (int)((uint32_t)slot - q * (uint32_t)kv.page_size)};
  } else {
    p.page = slot / kv.page_size;
    p.slot = (int)(slot - p.page * kv.page_size);
  }
  if (p.page >= kv.n_pages) {
    set_error(err, DEV_ERR_BOUNDS);
    return Place{-1, 0};
  }
  return p;
}

// One CTA per (token, block of rows): grid (T, row blocks).
template <int D>
__global__ void __launch_bounds__(kRowThreads) head_rows_kernel(const RowArgs a, int rows_per_cta) {
  constexpr int L = D / 8, kRows = kRowThreads / L;
  __shared__ float2 turn[D / 2];  // (cos, sin) of the token's angles
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % L, slot0 = threadIdx.x / L;
  const int n_rows = a.n_q + a.n_k + a.n_v;
  const int r0 = blockIdx.y * rows_per_cta;
  const int r1 = min(r0 + rows_per_cta, n_rows);
  if (a.half > 0) {
    const uint64_t pos = (uint64_t)(int64_t)a.positions[t];
    for (int i = threadIdx.x; i < a.half; i += kRowThreads) {
      // signed fraction of a turn in [-1/2, 1/2), as half turns for sincospi
      const float x = (float)(int64_t)(pos * a.turns[i]) * 0x1p-63f;
      float s, c;
      sincospif(x, &s, &c);
      turn[i] = make_float2(c, s);
    }
  }
  const Place at = a.cache ? place_of(a.slots[t], a.kv, a.err) : Place{-1, 0};
  __syncthreads();
  // every thread runs every iteration: the shuffles below take whole warps
  for (int base = r0; base < r1; base += kRows) {
    const int r = base + slot0;
    const bool on = r < r1;
    const bool is_q = r < a.n_q, is_k = !is_q && r < a.n_q + a.n_k;
    const int h = is_q ? r : (is_k ? r - a.n_q : r - a.n_q - a.n_k);
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (on) {
      const RowsIn &in = is_q ? a.q : (is_k ? a.k : a.v);
      unpack8(*reinterpret_cast<const uint4 *>(in.p + t * in.stride + h * D + lane * 8), y);
    }
    const float *w = is_q ? a.q_weight : (is_k ? a.k_weight : nullptr);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
    ss = row_sum<L>(ss);
    if (w != nullptr) {
      const float rms = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * rms * w[lane * 8 + i];
    }
    if (a.half > 0) {
      const int step = a.half / 8;  // lanes between the two halves
      const bool second = lane >= step;
      const int from = second ? lane - step : lane + step;
      float z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = __shfl_sync(0xffffffffu, y[i], from & (L - 1), L);
      if ((is_q || is_k) && lane * 8 < 2 * a.half) {
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 cs = turn[lane * 4 + i];
            const float u = y[2 * i], v = y[2 * i + 1];
            y[2 * i] = u * cs.x - v * cs.y;
            y[2 * i + 1] = v * cs.x + u * cs.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 cs = turn[(second ? lane - step : lane) * 8 + i];
            y[i] = second ? y[i] * cs.x + z[i] * cs.y : y[i] * cs.x - z[i] * cs.y;
          }
        }
      }
    }
    if (is_q || !a.cache) {
      if (on) {
        const RowsOut &o = is_q ? a.q_out : a.k_out;
        *reinterpret_cast<uint4 *>(o.p + t * o.stride + h * D + lane * 8) = pack8(y);
      }
      if (!a.cache || !a.e4m3) continue;
    }
    uint8_t *rows = is_k ? a.kv.k : a.kv.v;
    const int64_t off = at.page * a.kv.page_stride + h * a.kv.head_stride + at.slot * a.kv.slot_stride;
    const bool store = on && !is_q && at.page >= 0;
    if (!a.e4m3) {
      if (store) *reinterpret_cast<uint4 *>(rows + off + lane * 16) = pack8(y);
      continue;
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = fabsf(y[i]);
      if (m < INFINITY) amax = fmaxf(amax, m);
      else y[i] = NAN;  // an infinity has no code; a NaN stays one
    }
    amax = row_max<L>(amax);
    const int e = e4m3_row_exponent(amax);
    if (store) {
      const Pow2 down = pow2_factors(-e);
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(down(y[2 * i]), down(y[2 * i + 1])),
                                        __NV_SATFINITE, __NV_E4M3);
      *reinterpret_cast<uint2 *>(rows + off + lane * 8) =
          make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      if (lane == 0)
        (is_k ? a.kv.k_scale : a.kv.v_scale)[at.page * a.kv.scale_page_stride +
                                             h * a.kv.scale_head_stride +
                                             at.slot * a.kv.scale_slot_stride] = exp2i(e);
    }
  }
}

// Rows out of the cache: one CTA per token, a row's 8-element pieces over the
// lanes.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) read_rows_kernel(const ReadArgs a) {
  constexpr int L = D / 8, kRows = kRowThreads / L;
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % L, slot0 = threadIdx.x / L;
  const Place at = place_of(a.slots[t], a.kv, a.err);
  for (int r = slot0; r < 2 * a.n_kv; r += kRows) {
    const bool is_k = r < a.n_kv;
    const int h = is_k ? r : r - a.n_kv;
    uint4 o = make_uint4(0, 0, 0, 0);
    if (at.page >= 0) {
      const uint8_t *row = (is_k ? a.kv.k : a.kv.v) + at.page * a.kv.page_stride +
                           h * a.kv.head_stride + at.slot * a.kv.slot_stride;
      if (!E4M3) {
        o = *reinterpret_cast<const uint4 *>(row + lane * 16);
      } else {
        const float scale = (is_k ? a.kv.k_scale : a.kv.v_scale)[at.page * a.kv.scale_page_stride +
                                                                 h * a.kv.scale_head_stride +
                                                                 at.slot * a.kv.scale_slot_stride];
        const uint2 c = *reinterpret_cast<const uint2 *>(row + lane * 8);
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = unpack_f16x2(e4m3x2_to_f16x2((i < 2 ? c.x : c.y) >> (16 * (i & 1))));
          f[2 * i] = v.x * scale;
          f[2 * i + 1] = v.y * scale;
        }
        o = pack8(f);
      }
    }
    const RowsOut &out = is_k ? a.k_out : a.v_out;
    *reinterpret_cast<uint4 *>(out.p + t * out.stride + h * D + lane * 8) = o;
  }
}

template <int D>
cudaError_t rows_of(const RowArgs &a, cudaStream_t s) {
  const int n_rows = a.n_q + a.n_k + a.n_v;
  head_rows_kernel<D><<<dim3((unsigned)a.T, 1), kRowThreads, 0, s>>>(a, n_rows);
  return cudaGetLastError();
}

template <int D>
cudaError_t read_of(const ReadArgs &a, cudaStream_t s) {
  if (a.e4m3) read_rows_kernel<D, true><<<(unsigned)a.T, kRowThreads, 0, s>>>(a);
  else read_rows_kernel<D, false><<<(unsigned)a.T, kRowThreads, 0, s>>>(a);
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
