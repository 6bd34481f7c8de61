// C ABI of the operators around the layer in a training step: argument
// validation of the layer norm entry points.  The arithmetic is in
// layer_norm.cu.
#include <cmath>

#include "moe_kernels.cuh"

namespace moe {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool known_type(moe_dtype t) { return t == MOE_BF16 || t == MOE_FP32; }

moe_status check_norm_shape(int32_t T, int32_t D) {
  if (T < 0 || D <= 0) return MOE_ERR_INVALID_ARG;
  if (T > (1 << 24) || D > MOE_MAX_DIM) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_layer_norm_forward(const void* x, moe_dtype x_type, const void* add, const float* weight,
                                  const float* bias, float eps, int32_t T, int32_t D, void* y, void* h,
                                  float* mean, float* rstd, void* stream) {
  const moe_status st = check_norm_shape(T, D);
  if (st != MOE_OK) return st;
  if (!known_type(x_type) || !(eps >= 0.f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if ((add == nullptr) != (h == nullptr)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !weight || !y || !mean || !rstd) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {x, add, weight, bias, y, h, mean, rstd};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
  LayerNormArgs a{x, x_type == MOE_FP32, add, weight, bias, eps, T, D, y, h, mean, rstd};
  return cuda_status(launch_layer_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_layer_norm_backward_scratch_size(int32_t T, int32_t D) {
  if (check_norm_shape(T, D) != MOE_OK) return 0;
  const size_t rows = T < kLnMaxPartials ? T : kLnMaxPartials;
  return rows * 2 * D * sizeof(float);
}

moe_status moe_layer_norm_backward(const void* dy, const void* x, moe_dtype x_type, const float* weight,
                                   const float* mean, const float* rstd, const void* d_stream, int32_t T,
                                   int32_t D, void* dx, float* dweight, float* dbias, void* scratch,
                                   size_t scratch_bytes, void* stream) {
  const moe_status st = check_norm_shape(T, D);
  if (st != MOE_OK) return st;
  if (!known_type(x_type) || !dweight || !weight) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!dy || !x || !mean || !rstd || !dx || !scratch)) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {dy, x, weight, mean, rstd, d_stream, dx, dweight, dbias, scratch};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
  if (scratch_bytes < moe_layer_norm_backward_scratch_size(T, D)) return MOE_ERR_WORKSPACE;
  LayerNormBwdArgs a{dy, x, x_type == MOE_FP32, weight, mean, rstd, d_stream, T, D, dx, dweight, dbias,
                     static_cast<float*>(scratch)};
  return cuda_status(launch_layer_norm_bwd(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
