// Arithmetic that the attention's kernels share.
#pragma once

#include <cuda_runtime.h>

namespace fp8moe {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// tanh below 0.6: y + y^3 (t0 + t1 y^2 + ...), a least-squares fit of the relative
// error over Chebyshev points, 3e-9.
__device__ constexpr float kTanh[5] = {-0.33333298563957214f, 0.13331924378871918f, -0.053783830255270004f, 0.020795973017811775f,
                                       -0.005895158741623163f};

// tanh: the polynomial below 0.6, (1 - t) / (1 + t) with t = e^(-2|y|) above.
__device__ __forceinline__ float tanh_f32(float y) {
  const float z = y * y;
  float p = fmaf(z, kTanh[4], kTanh[3]);
  p = fmaf(z, p, kTanh[2]);
  p = fmaf(z, p, kTanh[1]);
  p = fmaf(z, p, kTanh[0]);
  const float small = fmaf(y * z, p, y);
  float t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(-2.f * kLog2e * fabsf(y)));
  const float large = copysignf(__fdividef(1.f - t, 1.f + t), y);
  return fabsf(y) < 0.6f ? small : large;
}

}  // namespace fp8moe
