// C ABI of the operators around the layer in a training step: argument
// validation of the layer norm and Newton-Schulz entry points.  The arithmetic
// is in layer_norm.cu, newton_schulz.cu and newton_schulz_small.cu.
#include <cmath>

#include <algorithm>

#include "moe_kernels.cuh"

namespace moe {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

bool known_type(moe_dtype t) { return t == MOE_BF16 || t == MOE_FP32; }

moe_status check_norm_shape(int32_t T, int32_t D) {
  if (T < 0 || D <= 0) return MOE_ERR_INVALID_ARG;
  if (T > (1 << 24) || D > MOE_MAX_DIM) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

moe_status check_matrix_shape(int32_t count, int32_t rows, int32_t cols) {
  if (count < 0 || rows <= 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
  if (count > MOE_MAX_MATRICES || rows > MOE_MAX_DIM || cols > MOE_MAX_DIM) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

// Steps, coefficients and eps into the problem.
moe_status set_steps(NsProblem* p, int32_t steps, const float* coefficients, float eps) {
  if (steps < 1 || !coefficients || !(eps >= 0.f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if (steps > MOE_MAX_NS_STEPS) return MOE_ERR_UNSUPPORTED_SHAPE;
  for (int i = 0; i < 3 * steps; ++i) {
    if (!std::isfinite(coefficients[i])) return MOE_ERR_INVALID_ARG;
    p->coeff[i / 3][i % 3] = coefficients[i];
  }
  p->steps = steps;
  p->eps = eps;
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

size_t moe_newton_schulz_workspace_size(int32_t count, int32_t rows, int32_t cols) {
  if (check_matrix_shape(count, rows, cols) != MOE_OK) return 0;
  return ns_workspace_bytes(count, std::min(rows, cols), std::max(rows, cols));
}

moe_status moe_newton_schulz(const void* grad, moe_dtype grad_type, int32_t count, int32_t rows, int32_t cols,
                             int32_t steps, const float* coefficients, float eps, void* out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  moe_status st = check_matrix_shape(count, rows, cols);
  if (st != MOE_OK) return st;
  NsProblem p{};
  if (!known_type(grad_type)) return MOE_ERR_INVALID_ARG;
  if ((st = set_steps(&p, steps, coefficients, eps)) != MOE_OK) return st;
  if (count == 0) return MOE_OK;
  if (!grad || !out || !workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned16(grad) || !aligned16(out) || !aligned256(workspace)) return MOE_ERR_INVALID_ARG;
  p.count = count;
  p.m = std::min(rows, cols);
  p.n = std::max(rows, cols);
  if (workspace_bytes < ns_workspace_bytes(count, p.m, p.n)) return MOE_ERR_WORKSPACE;
  p.grad_fp32 = grad_type == MOE_FP32;
  p.out.kind = kNsPlain;
  p.stacks.n = 1;
  p.stacks.s[0] = NsStack{grad, nullptr, out, nullptr, 0, rows > cols};
  return cuda_status(launch_newton_schulz(p, workspace, static_cast<cudaStream_t>(stream)));
}

moe_status moe_muon_step(const moe_matrix_stack* stacks, int32_t n_stacks, moe_dtype grad_type,
                         moe_dtype weight_type, const moe_muon_params* params, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (n_stacks < 0 || (n_stacks > 0 && !stacks) || !params) return MOE_ERR_INVALID_ARG;
  if (n_stacks > MOE_MAX_STACKS) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!known_type(grad_type) || !known_type(weight_type)) return MOE_ERR_INVALID_ARG;
  const moe_muon_params& q = *params;
  for (float v : {q.lr, q.momentum, q.weight_decay, q.scale})
    if (!std::isfinite(v)) return MOE_ERR_INVALID_ARG;
  if (q.nesterov != 0 && q.nesterov != 1) return MOE_ERR_INVALID_ARG;
  NsProblem p{};
  moe_status st = set_steps(&p, q.steps, q.coefficients, q.eps);
  if (st != MOE_OK) return st;
  for (int i = 0; i < n_stacks; ++i) {
    const moe_matrix_stack& k = stacks[i];
    if ((st = check_matrix_shape(k.count, k.rows, k.cols)) != MOE_OK) return st;
    const int m = std::min(k.rows, k.cols), n = std::max(k.rows, k.cols);
    if (i == 0) p.m = m, p.n = n;
    if (m != p.m || n != p.n) return MOE_ERR_INVALID_ARG;
    if (k.count == 0) continue;
    if (!k.weight || !k.grad || !k.momentum) return MOE_ERR_INVALID_ARG;
    if (k.weight_bf16 && weight_type != MOE_FP32) return MOE_ERR_INVALID_ARG;
    const void* ptrs[] = {k.weight, k.grad, k.momentum, k.weight_bf16};
    for (const void* v : ptrs)
      if (!aligned16(v)) return MOE_ERR_INVALID_ARG;
    p.stacks.s[p.stacks.n++] = NsStack{k.grad, k.momentum, k.weight, k.weight_bf16, p.count, k.rows > k.cols};
    p.count += k.count;
    if (p.count > MOE_MAX_MATRICES) return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  if (p.count == 0) return MOE_OK;
  if (!workspace || !aligned256(workspace)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < ns_workspace_bytes(p.count, p.m, p.n)) return MOE_ERR_WORKSPACE;
  p.grad_fp32 = grad_type == MOE_FP32;
  p.momentum = q.momentum;
  p.nesterov = q.nesterov;
  p.out.kind = weight_type == MOE_FP32 ? kNsWeightF32 : kNsWeightBf16;
  p.out.keep = static_cast<float>(1.0 - static_cast<double>(q.lr) * q.weight_decay);
  p.out.step = q.lr * q.scale;
  return cuda_status(launch_newton_schulz(p, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
