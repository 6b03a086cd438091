// Arithmetic that the attention's kernels share.
#pragma once

#include <cuda_runtime.h>

namespace fp8moe {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// tanh: an odd polynomial below 0.6 (least-squares fit of the relative error
// over Chebyshev points, 3e-9), (1 - t) / (1 + t) with t = e^(-2|y|) above.
__device__ __forceinline__ float tanh_f32(float y) {
  const float z = y * y;
  float p = fmaf(z, -0.005895158741623163f, 0.020795973017811775f);
  p = fmaf(z, p, -0.053783830255270004f);
  p = fmaf(z, p, 0.13331924378871918f);
  p = fmaf(z, p, -0.33333298563957214f);
  const float small = fmaf(y * z, p, y);
  float t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(-2.f * kLog2e * fabsf(y)));
  const float large = copysignf(__fdividef(1.f - t, 1.f + t), y);
  return fabsf(y) < 0.6f ? small : large;
}

}  // namespace fp8moe
