// Attention of one new token per sequence over a paged key/value cache
// (moe_attn_decode).
//
// out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), with the running maximum m
// and sum of one pass over the keys: when m grows, what was summed so far is
// scaled by e^(m_old - m_new).  One CTA per (query head, sequence); a warp
// takes every fourth key, a lane d / 32 elements of it, and the four warps'
// states are joined in shared memory.
#include "common.cuh"
#include "paged_attn.h"

namespace fp8moe {

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) decode_kernel(const DecodeArgs a) {
  constexpr int E = D / 32;
  __shared__ float acc_s[kWarps][D], m_s[kWarps], l_s[kWarps];
  const int b = blockIdx.x, h = blockIdx.y, c = h / (a.n_heads / a.n_kv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t len = a.lens[b];
  if (len < 0 || len > a.capacity) {
    set_error(a.err, DEV_ERR_BOUNDS);
    len = len < 0 ? 0 : a.capacity;
  }
  int64_t lo = a.starts ? a.starts[b] : 0;
  if (lo < 0) lo = 0;
  if (a.window > 0 && lo < len - a.window) lo = len - a.window;
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  float q[E], acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = __bfloat162float(a.q[(int64_t)b * a.q_stride + h * D + lane * E + i]);
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t j = lo + warp; j < len; j += kWarps) {
    const int64_t page = a.table[(int64_t)b * a.table_stride + j / a.kv.page_size];
    const int64_t slot = j % a.kv.page_size;
    float kf[E], vf[E];
    if (page < 0 || page >= a.kv.n_pages) {
      set_error(a.err, DEV_ERR_BOUNDS);
#pragma unroll
      for (int i = 0; i < E; ++i) kf[i] = vf[i] = 0.f;
    } else {
      const int64_t off = page * a.kv.page_stride + c * a.kv.head_stride + slot * a.kv.slot_stride;
      if (E4M3) {
        const int64_t so = page * a.kv.scale_page_stride + c * a.kv.scale_head_stride +
                           slot * a.kv.scale_slot_stride;
        const float ks = a.kv.k_scale[so], vs = a.kv.v_scale[so];
#pragma unroll
        for (int i = 0; i < E; ++i) {
          kf[i] = unpack_f16x2(e4m3x2_to_f16x2(a.kv.k[off + lane * E + i])).x * ks;
          vf[i] = unpack_f16x2(e4m3x2_to_f16x2(a.kv.v[off + lane * E + i])).x * vs;
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          kf[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.kv.k + off)[lane * E + i]);
          vf[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.kv.v + off)[lane * E + i]);
        }
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], kf[i], s);
    s = warp_sum(s) * a.scale;
    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    s = fmaf(slope, (float)(j - (len - 1)), s) * kLog2e;
    const float mn = fmaxf(m, s);
    const float keep = m == -INFINITY ? 1.f : exp2f(m - mn);
    const float p = exp2f(s - (mn == -INFINITY ? 0.f : mn));
    l = l * keep + p;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = fmaf(p, vf[i], acc[i] * keep);
    m = mn;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) acc_s[warp][lane * E + i] = acc[i];
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  __syncthreads();
  float mx = -INFINITY;
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, m_s[w]);
  float f[kWarps], sum = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    // a state without keys holds zeros, or NaN, whatever its factor
    f[w] = m_s[w] == -INFINITY ? 1.f : exp2f(m_s[w] - mx);
    sum += f[w] * l_s[w];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t bh = (int64_t)b * a.n_heads + h;
  for (int i = threadIdx.x; i < D; i += 32 * kWarps) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w) o += f[w] * acc_s[w][i];
    a.out[bh * D + i] = __float2bfloat16_rn(o * inv);
  }
  if (a.lse && threadIdx.x == 0) a.lse[bh] = (mx + log2f(sum)) * kLn2;
}

template <int D>
cudaError_t decode_of(const DecodeArgs &a, bool e4m3, cudaStream_t s) {
  const dim3 grid((unsigned)a.B, (unsigned)a.n_heads);
  if (e4m3) decode_kernel<D, true><<<grid, 32 * kWarps, 0, s>>>(a);
  else decode_kernel<D, false><<<grid, 32 * kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_decode(const DecodeArgs &a, int d, bool e4m3, cudaStream_t s) {
  switch (d) {
    case 64: return decode_of<64>(a, e4m3, s);
    case 128: return decode_of<128>(a, e4m3, s);
    case 256: return decode_of<256>(a, e4m3, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fp8moe
