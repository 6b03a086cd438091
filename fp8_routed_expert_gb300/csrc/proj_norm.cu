// Hidden-state rows of a block: the residual's addition, the RMS norm and the
// quantisation to e4m3 with a scale for each 128 columns, in one pass
// (moe_proj_norm of the C ABI).
//
// Per row of H columns, in f32:
//   r' = bf16(x + residual), written back: the rounded sum is the residual stream,
//        and the norm is of what later layers will add to
//   y  = r' / sqrt(mean(r'^2) + eps) * weight
//   out = bf16(y);  scale_b = max|y| / 448 over block b, code = e4m3(y / scale_b)
//
// Every byte is read once and written once, so HBM bounds it; a row's values stay
// in registers between the sum of squares and the outputs.  A row belongs to a
// group of `Group` lanes, lane i taking the 16-byte vectors i, i + Group, ...: 16
// neighbouring lanes hold the 128 columns of a block, whose largest value is four
// shuffles away.  A CTA keeps its columns' weights in registers over its rows, and
// the next row's loads are issued before this row is finished.
//
// 4096 rows of 6144, with residual, bf16 and e4m3 outputs: 38 us, 5.97 TB/s, 88% of the
// measured copy rate (issue slots 48%); 2048 rows of 16384 6.0 TB/s.  One row of 2048 takes
// 1.65 us, which is a launch with one chain of loads and one of shuffles.
#include "common.cuh"
#include "kernels.h"
#include "proj.h"
#include "tcgen05_ops.cuh"

namespace fp8moe {
using namespace sm100;
namespace {

constexpr int kCta = 256;  // threads, unless a row takes more

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint4 *>(p); }

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = u4_word(v, i);
    f[2 * i] = __uint_as_float(w << 16);
    f[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// A row's sum of squares is out of the range where f32 holds it to all its bits:
// above 2^120 (infinite and NaN ones too), or below 2^-90 where eps does not
// outweigh it.
__device__ __forceinline__ bool beyond(float ss, float eps) { return !(ss <= 0x1p120f) || (ss < 0x1p-90f && eps < 0x1p-90f); }

// Quotients y / s to f32 for s from 2^-90 on, rounded once as a division's are (those
// below 2^-10, whose code is zero, may be off by a unit).  Times the rounded inverse
// alone, values next to a tie of two codes go to the other one, a code in 2000.  Markstein
// (1990): a quotient within a unit, corrected by its residual times the correctly rounded
// inverse, is the rounded one; the first product may be off by 1.5 units, so it is
// corrected twice.  4096 rows of 6144 take 38.1 us as without (777 of 2880 4.9, so 4.5); a
// division each takes 42.4 (8.7).  Zeros keep their sign, and an infinity becomes a NaN, as
// the format has none.
struct Divisor {
  uint64_t s, inv, minus;
  __device__ __forceinline__ explicit Divisor(float v) : s(pack_f32x2(v, v)) {
    const float i = 1.f / v;
    inv = pack_f32x2(i, i);
    minus = pack_f32x2(-i, -i);
  }
  __device__ __forceinline__ float2 quotients(float y0, float y1) const {
    const uint64_t y = pack_f32x2(-y0, -y1);
    uint64_t q = mul_f32x2(pack_f32x2(y0, y1), inv);
    q = fma_f32x2(fma_f32x2(q, s, y), minus, q);
    q = fma_f32x2(fma_f32x2(q, s, y), minus, q);
    return unpack_f32x2(q);
  }
};

// Sum over the group's lanes, the same bits in each.  Groups of more than a warp
// pass the CTA's barrier once; *odd tells, alike for all that share a barrier,
// whether one of their sums is beyond.
template <int Group, int Threads>
__device__ __forceinline__ float group_sum(float v, float *part, float eps, bool *odd) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (Group == 32) {
    *odd = beyond(v, eps);
    return v;
  } else {
    constexpr int kWarps = Group / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    *odd = false;
#pragma unroll
    for (int g = 0; g < Threads / Group; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) sum += part[g * kWarps + i];
      *odd |= beyond(sum, eps);
      if (g == warp / kWarps) v = sum;
    }
    return v;
  }
}

template <int Group, int Vecs>
__global__ void __launch_bounds__(Group > kCta ? Group : kCta) norm_kernel(const NormArgs a) {
  constexpr int kThreads = Group > kCta ? Group : kCta, kRows = kThreads / Group;
  __shared__ float part[3][kThreads / 32];
  const int in_group = threadIdx.x % Group, group = threadIdx.x / Group;
  const int vecs = a.H / 8;
  pdl_wait();
  pdl_trigger();
  float w[Vecs][8];
#pragma unroll
  for (int i = 0; i < Vecs; ++i) {
    const int v = in_group + i * Group;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
      if (a.weight != nullptr && v < vecs) f = __ldg(reinterpret_cast<const float4 *>(a.weight + 8 * v + j));
      w[i][j] = f.x, w[i][j + 1] = f.y, w[i][j + 2] = f.z, w[i][j + 3] = f.w;
    }
  }
  uint4 xn[Vecs], rn[Vecs];
  const auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < Vecs; ++i) {
      const int v = in_group + i * Group;
      xn[i] = rn[i] = make_uint4(0u, 0u, 0u, 0u);
      if (t < a.T && v < vecs) {
        xn[i] = ld16(a.x + t * a.x_stride + 8 * v);
        if (a.residual != nullptr) rn[i] = ld16(a.residual + t * a.residual_stride + 8 * v);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t t = (int64_t)blockIdx.x * kRows + group;
  load(t);
  int turn = 0;
  // every group of a CTA takes the same number of turns: its barriers are the CTA's
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.T; base += step, t += step) {
    float y[Vecs][8];
#pragma unroll
    for (int i = 0; i < Vecs; ++i) unpack8(xn[i], y[i]);
    if (a.residual != nullptr) {
#pragma unroll
      for (int i = 0; i < Vecs; ++i) {
        float r[8];
        unpack8(rn[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] += r[j];
        const uint4 s = pack8(y[i]);
        const int v = in_group + i * Group;
        if (t < a.T && v < vecs) *reinterpret_cast<uint4 *>(a.residual_out + t * a.residual_out_stride + 8 * v) = s;
        unpack8(s, y[i]);
      }
    }
    load(t + step);
    if (a.weight != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < Vecs; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[i][j], y[i][j], ss);
      bool odd;
      ss = group_sum<Group, kThreads>(ss, part[turn], a.eps, &odd);
      const float n = 1.f / (float)a.H;
      float eps = a.eps;
      if (odd) {  // rows beyond are normed at a power of two that brings them back
        const float pre = !beyond(ss, eps) ? 1.f : ss < 1.f ? 0x1p64f : 0x1p-72f;
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < Vecs; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            y[i][j] *= pre;
            ss = fmaf(y[i][j], y[i][j], ss);
          }
        ss = group_sum<Group, kThreads>(ss, part[2], a.eps, &odd);
        eps = a.eps * pre * pre;
      }
      const float r = rsqrtf(fmaf(ss, n, eps));
      // the normed value first: 1 / rms times a weight may leave f32 where the output does not
#pragma unroll
      for (int i = 0; i < Vecs; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] = y[i][j] * r * w[i][j];
    }
    turn ^= 1;
    if (t < a.T) {
#pragma unroll
      for (int i = 0; i < Vecs; ++i) {
        const int v = in_group + i * Group;
        if (a.out != nullptr && v < vecs) *reinterpret_cast<uint4 *>(a.out + t * a.out_stride + 8 * v) = pack8(y[i]);
      }
    }
    if (a.codes != nullptr) {
#pragma unroll
      for (int i = 0; i < Vecs; ++i) {
        const int v = in_group + i * Group;
        // the scale comes from the block's finite values
        float am = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float m = fabsf(y[i][j]);
          am = fmaxf(am, m <= 3.402823466e38f ? m : 0.f);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        // a scale is a normal number, so that its inverse is one too
        const float scale = am > 0.f ? fmaxf(am / 448.f, 0x1p-126f) : 1.f;
        float divisor = scale;
        if (scale < 0x1p-90f) {  // residuals below would leave f32: y and the divisor at 2^64 times their size
          divisor *= 0x1p64f;
#pragma unroll
          for (int j = 0; j < 8; ++j) y[i][j] *= 0x1p64f;
        }
        const Divisor by(divisor);
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          c[j] = __nv_cvt_float2_to_fp8x2(by.quotients(y[i][2 * j], y[i][2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
        if (t < a.T && v < vecs) {
          *reinterpret_cast<uint2 *>(a.codes + t * a.codes_stride + 8 * v) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
          if ((v & 15) == 0) a.scales[t * a.scale_row + (v >> 4) * a.scale_block] = scale;
        }
      }
    }
  }
}

template <int Group, int Vecs>
cudaError_t launch_one(const NormArgs &a, int sms, int limit, cudaStream_t s) {
  constexpr int kThreads = Group > kCta ? Group : kCta, kRows = kThreads / Group;
  static const int resident = [] {
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_kernel<Group, Vecs>, kThreads, 0) == cudaSuccess && n > 0 ? n : 1;
  }();
  // with a limit a CTA per SM: more than one would go to an SM each while others are idle
  const int64_t ctas = (a.T + kRows - 1) / kRows, most = limit > 0 ? limit : (int64_t)sms * resident;
  return launch_pdl(norm_kernel<Group, Vecs>, dim3((unsigned)(ctas < most ? ctas : most)), dim3(kThreads), 0, s, a);
}

template <int Group>
cudaError_t launch_group(const NormArgs &a, int vecs, int sms, int limit, cudaStream_t s) {
  switch (vecs) {
    case 1: return launch_one<Group, 1>(a, sms, limit, s);
    case 2: return launch_one<Group, 2>(a, sms, limit, s);
    case 3: return launch_one<Group, 3>(a, sms, limit, s);
    default: return launch_one<Group, 4>(a, sms, limit, s);
  }
}

}  // namespace

// Lanes of a row and vectors of a lane: as few idle lanes as may be, and then as many
// lanes, which hold less each (one row of 2048 by 256 lanes 1.65 us, by 64 lanes of four
// vectors 2.9).  The grid is what is resident: more CTAs than that load their weights
// again (777 rows of 2880 5.1 us, so 4.6).
cudaError_t launch_norm(const NormArgs &a, int sms, int limit, cudaStream_t s) {
  const int vecs = a.H / 8;
  int group = 0, per = 0;
  for (int v = 1; v <= 4; ++v) {
    int g = 32;
    while (g < 512 && g * v < vecs) g *= 2;
    if (g * v >= vecs && (group == 0 || g * v < group * per)) group = g, per = v;
  }
  switch (group) {
    case 32: return launch_group<32>(a, per, sms, limit, s);
    case 64: return launch_group<64>(a, per, sms, limit, s);
    case 128: return launch_group<128>(a, per, sms, limit, s);
    case 256: return launch_group<256>(a, per, sms, limit, s);
    default: return launch_group<512>(a, per, sms, limit, s);
  }
}

}  // namespace fp8moe
