// C ABI of the projections: context, argument checks and launches.  See
// include/fp8moe.h for the contract.
#include <cmath>
#include <new>

#include "common.cuh"
#include "fp8moe.h"
#include "proj.h"
#include "tensor_map.h"

using namespace fp8moe;

struct moe_proj {
  int device = 0, sms = 0;
  int limit = 0;  // SMs that a call may fill, 0 for all
  MatmulFit fit{};
  int *err = nullptr;
  cudaStream_t last_stream = nullptr;
};

namespace {

#define PROJ_TRY(x)                              \
  do {                                           \
    if ((x) != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)
#define CHECK(x)                   \
  do {                             \
    const int rc_ = (x);           \
    if (rc_ != MOE_OK) return rc_; \
  } while (0)

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxRows = INT64_C(0x7fffffff), kMaxSide = INT64_C(0x7fffff00), kMaxStride = INT64_C(1) << 31;

// Rows of `columns` elements of `bytes` each, whose starts are `align` bytes apart.
int check_rows(const void *p, int64_t stride, int64_t columns, int bytes, int align) {
  if (p == nullptr) return MOE_ERR_ARG;
  if (stride < columns || stride > kMaxStride) return MOE_ERR_SHAPE;
  if (!aligned(p, (size_t)align) || stride * bytes % align != 0) return MOE_ERR_ALIGN;
  return MOE_OK;
}

int check_scales(const void *p, int64_t row, int64_t block) {
  if (p == nullptr) return MOE_ERR_ARG;
  if (row < 1 || block < 1 || row > kMaxStride || block > kMaxStride) return MOE_ERR_SHAPE;
  return aligned(p, 4) ? MOE_OK : MOE_ERR_ALIGN;
}

}  // namespace

extern "C" {

int moe_proj_init(moe_proj **out, int32_t device, int32_t max_sms) {
  if (out == nullptr) return MOE_ERR_ARG;
  *out = nullptr;
  if (device < 0 || max_sms < 0) return MOE_ERR_SHAPE;
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || device >= count) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  PROJ_TRY(cudaSetDevice(device));
  int major = 0, minor = 0, sms = 0;
  PROJ_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device));
  PROJ_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device));
  PROJ_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device));
  if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED;
  MatmulFit fit{};
  PROJ_TRY(ready_matmul(&fit));
  moe_proj *p = new (std::nothrow) moe_proj();
  if (p == nullptr) return MOE_ERR_NOMEM;
  p->device = device;
  p->fit = fit;
  p->sms = sms;
  p->limit = max_sms < sms ? max_sms : 0;
  if (cudaMalloc(&p->err, 256) != cudaSuccess) {
    cudaGetLastError();
    delete p;
    return MOE_ERR_NOMEM;
  }
  // ready for any stream when this returns
  if (cudaMemset(p->err, 0, 256) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    moe_proj_free(p);
    return MOE_ERR_CUDA;
  }
  *out = p;
  return MOE_OK;
}

void moe_proj_free(moe_proj *p) {
  if (p == nullptr) return;
  cudaSetDevice(p->device);
  if (p->err) cudaFree(p->err);
  delete p;
}

int moe_proj_status(moe_proj *p) {
  if (p == nullptr) return MOE_ERR_ARG;
  PROJ_TRY(cudaSetDevice(p->device));
  PROJ_TRY(cudaStreamSynchronize(p->last_stream));
  int flag = 0;
  PROJ_TRY(cudaMemcpy(&flag, p->err, sizeof(int), cudaMemcpyDeviceToHost));
  PROJ_TRY(cudaMemset(p->err, 0, sizeof(int)));
  // a kernel on a stream that does not wait for the default one must find it cleared
  PROJ_TRY(cudaStreamSynchronize(nullptr));
  return flag ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}

int moe_proj_norm(moe_proj *p, const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                  int64_t T, int64_t H, const float *weight, float eps, void *residual_out,
                  int64_t residual_out_stride, void *out, int64_t out_stride, uint8_t *codes, int64_t codes_stride,
                  float *scales, int64_t scale_row_stride, int64_t scale_block_stride, void *stream) {
  if (p == nullptr || T < 0) return MOE_ERR_ARG;
  if (T > kMaxRows || H < 8 || H > kNormColumns || H % 8 != 0) return MOE_ERR_SHAPE;
  if (!std::isfinite(eps) || eps < 0.f) return MOE_ERR_ARG;
  if ((residual == nullptr) != (residual_out == nullptr) || (codes == nullptr) != (scales == nullptr)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (out == nullptr && codes == nullptr && residual == nullptr) return MOE_ERR_ARG;
  CHECK(check_rows(x, x_stride, H, 2, 16));
  if (residual != nullptr) {
    CHECK(check_rows(residual, residual_stride, H, 2, 16));
    CHECK(check_rows(residual_out, residual_out_stride, H, 2, 16));
  }
  if (out != nullptr) CHECK(check_rows(out, out_stride, H, 2, 16));
  if (codes != nullptr) {
    CHECK(check_rows(codes, codes_stride, H, 1, 8));
    CHECK(check_scales(scales, scale_row_stride, scale_block_stride));
  }
  if (!aligned(weight, 16)) return MOE_ERR_ALIGN;
  NormArgs a{};
  a.x = static_cast<const __nv_bfloat16 *>(x);
  a.x_stride = x_stride;
  a.residual = static_cast<const __nv_bfloat16 *>(residual);
  a.residual_stride = residual_stride;
  a.T = T;
  a.H = (int)H;
  a.weight = weight;
  a.eps = eps;
  a.residual_out = static_cast<__nv_bfloat16 *>(residual_out);
  a.residual_out_stride = residual_out_stride;
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.out_stride = out_stride;
  a.codes = codes;
  a.codes_stride = codes_stride;
  a.scales = scales;
  a.scale_row = scale_row_stride;
  a.scale_block = scale_block_stride;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  PROJ_TRY(cudaSetDevice(p->device));
  p->last_stream = s;
  PROJ_TRY(launch_norm(a, p->sms, p->limit, s));
  return MOE_OK;
}

int moe_proj_matmul(moe_proj *p, const uint8_t *a, int64_t a_stride, const float *a_scale, int64_t scale_row_stride,
                    int64_t scale_block_stride, int64_t M, const uint8_t *w, int64_t w_stride, const float *w_scale,
                    int64_t N, int64_t K, void *out, int64_t out_stride, void *stream) {
  if (p == nullptr || M < 0 || N < 0 || K < 0) return MOE_ERR_ARG;
  if (M > kMaxSide || N > kMaxSide || K > kMaxSide) return MOE_ERR_SHAPE;
  if (M == 0 || N == 0) return MOE_OK;
  CHECK(check_rows(out, out_stride, N, 2, 16));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) {
    PROJ_TRY(cudaSetDevice(p->device));
    p->last_stream = s;
    PROJ_TRY(cudaMemset2DAsync(out, (size_t)out_stride * 2, 0, (size_t)N * 2, (size_t)M, s));
    return MOE_OK;
  }
  CHECK(check_rows(a, a_stride, K, 1, 16));
  CHECK(check_rows(w, w_stride, K, 1, 16));
  CHECK(check_scales(a_scale, scale_row_stride, scale_block_stride));
  CHECK(check_scales(w_scale, 1, 1));
  MatmulArgs m{};
  m.M = M;
  m.N = N;
  m.K = K;
  m.a_scale = a_scale;
  m.a_row = scale_row_stride;
  m.a_block = scale_block_stride;
  m.w_scale = w_scale;
  m.out = static_cast<__nv_bfloat16 *>(out);
  m.out_stride = out_stride;
  m.whole_lines = aligned(out, 32) && out_stride % 16 == 0;
  m.blocks = (int)((K + 127) / 128);
  m.err = p->err;
  plan_matmul(p->fit, p->sms, p->limit, &m);
  CUtensorMap ta, tw, to;
  const uint64_t a_sizes[2] = {(uint64_t)K, (uint64_t)M}, a_strides[1] = {(uint64_t)a_stride};
  const uint64_t w_sizes[2] = {(uint64_t)K, (uint64_t)N}, w_strides[1] = {(uint64_t)w_stride};
  const uint64_t o_sizes[2] = {(uint64_t)(N & ~INT64_C(7)), (uint64_t)M}, o_strides[1] = {(uint64_t)out_stride * 2};
  const uint32_t a_box[2] = {128, (uint32_t)m.a_rows}, w_box[2] = {128, (uint32_t)m.columns}, o_box[2] = {64, 32};
  PROJ_TRY(cudaSetDevice(p->device));
  if (!encode_tile_map(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a, a_sizes, a_strides, a_box) ||
      !encode_tile_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, w, w_sizes, w_strides, w_box))
    return MOE_ERR_CUDA;
  if (m.columns < 256) to = tw;  // (only the widest tiles' outputs leave by TMA, N well above 8)
  else if (!encode_tile_map(&to, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, o_sizes, o_strides, o_box)) return MOE_ERR_CUDA;
  p->last_stream = s;
  PROJ_TRY(launch_matmul(ta, tw, to, m, s));
  return MOE_OK;
}

}  // extern "C"
