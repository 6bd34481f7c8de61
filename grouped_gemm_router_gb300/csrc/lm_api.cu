// C ABI of the ends of a language model: argument validation of the embedding,
// cross entropy and distillation entry points.  The arithmetic is in
// embedding.cu and vocab_head.cu.
#include <cmath>
#include <initializer_list>

#include "moe_kernels.cuh"

namespace moe {
namespace {

bool on(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool all_on_16(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!on(p, 16)) return false;
  return true;
}

bool all_there(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!p) return false;
  return true;
}

bool known_type(moe_dtype t) { return t == MOE_BF16 || t == MOE_FP32; }
bool known_index(moe_index_type t) { return t == MOE_I32 || t == MOE_I64; }

moe_status check_table(int32_t T, int32_t V, int32_t D) {
  if (T < 0 || V <= 0 || D <= 0) return MOE_ERR_INVALID_ARG;
  if (T > (1 << 24) || V > MOE_MAX_VOCAB || D > MOE_MAX_DIM) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

moe_status check_head(int32_t T, int32_t D, int32_t V) {
  const moe_status st = check_table(T, V, D);
  if (st != MOE_OK) return st;
  return D % 64 == 0 ? MOE_OK : MOE_ERR_UNSUPPORTED_SHAPE;
}

moe_status check_teacher(const moe_teacher* t, int32_t T) {
  if (!t || !known_index(t->ids_type) || !known_type(t->logits_type)) return MOE_ERR_INVALID_ARG;
  // (the kernels multiply by log2(e) / temperature)
  if (t->K < 1 || !(t->temperature > 0.f) || !std::isfinite(t->temperature) || !std::isfinite(2.f / t->temperature))
    return MOE_ERR_INVALID_ARG;
  if (t->K > MOE_MAX_TEACHER) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T > 0 && !all_there({t->ids, t->logits})) return MOE_ERR_INVALID_ARG;
  return all_on_16({t->ids, t->logits}) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

moe_status check_workspace(const void* workspace, size_t bytes, size_t needed) {
  if (!workspace || !on(workspace, 256)) return MOE_ERR_INVALID_ARG;
  return bytes < needed ? MOE_ERR_WORKSPACE : MOE_OK;
}

VocabTargets targets_of(const moe_teacher& t) {
  return VocabTargets{t.ids, t.ids_type == MOE_I64, t.K, t.logits, t.logits_type == MOE_FP32};
}

// T = 0 leaves nothing but a weight gradient of zeros.
moe_status zero_weight_gradient(void* dW, int32_t V, int32_t D, cudaStream_t s) {
  return cuda_status(cudaMemsetAsync(dW, 0, static_cast<size_t>(V) * D * 2, s));
}

moe_status embedding_backward(const void* d_out, moe_dtype d_type, const void* ids, moe_index_type ids_type,
                              float scale, const void* add, int32_t T, int32_t V, int32_t D, float* d_table,
                              void* scratch, size_t scratch_bytes, void* stream, int by_passes) {
  const moe_status st = check_table(T, V, D);
  if (st != MOE_OK) return st;
  if (!known_index(ids_type) || !known_type(d_type) || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (!d_table || (T > 0 && !all_there({d_out, ids}))) return MOE_ERR_INVALID_ARG;
  if (!all_on_16({d_out, ids, add, d_table})) return MOE_ERR_INVALID_ARG;
  const moe_status ws = check_workspace(scratch, scratch_bytes, embedding_bwd_scratch_bytes(T, V, D));
  if (ws != MOE_OK) return ws;
  EmbeddingBwdArgs a{d_out, d_type == MOE_FP32, ids, ids_type == MOE_I64, scale, add, T, V, D, d_table, by_passes};
  return cuda_status(launch_embedding_bwd(a, scratch, static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_embedding_forward(const void* ids, moe_index_type ids_type, const void* table, moe_dtype table_type,
                                 float scale, int32_t T, int32_t V, int32_t D, void* out, moe_dtype out_type,
                                 void* stream) {
  const moe_status st = check_table(T, V, D);
  if (st != MOE_OK) return st;
  if (!known_index(ids_type) || !known_type(table_type) || !known_type(out_type) || !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!all_there({ids, table, out}) || !all_on_16({ids, table, out})) return MOE_ERR_INVALID_ARG;
  EmbeddingArgs a{ids, ids_type == MOE_I64, table, table_type == MOE_FP32, scale, T, V, D, out, out_type == MOE_FP32};
  return cuda_status(launch_embedding(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_embedding_backward_scratch_size(int32_t T, int32_t V, int32_t D) {
  return check_table(T, V, D) != MOE_OK ? 0 : embedding_bwd_scratch_bytes(T, V, D);
}

moe_status moe_embedding_backward(const void* d_out, moe_dtype d_type, const void* ids, moe_index_type ids_type,
                                  float scale, const void* add, int32_t T, int32_t V, int32_t D, float* d_table,
                                  void* scratch, size_t scratch_bytes, void* stream) {
  return embedding_backward(d_out, d_type, ids, ids_type, scale, add, T, V, D, d_table, scratch, scratch_bytes, stream, 0);
}

moe_status moe_selftest_embedding_by_passes(const void* d_out, moe_dtype d_type, const void* ids,
                                            moe_index_type ids_type, float scale, const void* add, int32_t T, int32_t V,
                                            int32_t D, float* d_table, void* scratch, size_t scratch_bytes,
                                            void* stream) {
  return embedding_backward(d_out, d_type, ids, ids_type, scale, add, T, V, D, d_table, scratch, scratch_bytes, stream, 1);
}

size_t moe_vocab_forward_workspace_size(int32_t T, int32_t D, int32_t V, int32_t n_teacher) {
  if (check_head(T, D, V) != MOE_OK || n_teacher < 0 || n_teacher > MOE_MAX_TEACHER) return 0;
  return vocab_forward_workspace_bytes(T, D, V, n_teacher);
}

size_t moe_vocab_backward_workspace_size(int32_t T, int32_t D, int32_t V, int32_t n_teacher) {
  if (check_head(T, D, V) != MOE_OK || n_teacher < 0 || n_teacher > MOE_MAX_TEACHER) return 0;
  return vocab_backward_workspace_bytes(T, D, V, n_teacher);
}

moe_status moe_cross_entropy_forward(const void* x, const void* W, const void* labels, moe_index_type labels_type,
                                     int32_t T, int32_t D, int32_t V, float* loss, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  moe_status st = check_head(T, D, V);
  if (st != MOE_OK) return st;
  if (!known_index(labels_type)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!all_there({x, W, labels, loss, lse}) || !all_on_16({x, W, labels, loss, lse})) return MOE_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes, vocab_forward_workspace_bytes(T, D, V, 0))) != MOE_OK) return st;
  VocabForward a{x, W, VocabTargets{labels, labels_type == MOE_I64, 0, nullptr, 0}, 1.f, T, D, V, loss, lse, nullptr};
  return cuda_status(launch_vocab_forward(a, workspace, static_cast<cudaStream_t>(stream)));
}

moe_status moe_cross_entropy_backward(const float* d_loss, const float* d_lse, const void* x, const void* W,
                                      const void* labels, moe_index_type labels_type, const float* loss,
                                      const float* lse, int32_t T, int32_t D, int32_t V, void* dx, void* dW,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  moe_status st = check_head(T, D, V);
  if (st != MOE_OK) return st;
  if (!known_index(labels_type) || !dW || !on(dW, 16)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) return zero_weight_gradient(dW, V, D, s);
  if (!all_there({d_loss, x, W, labels, loss, lse, dx})) return MOE_ERR_INVALID_ARG;
  if (!all_on_16({d_loss, d_lse, x, W, labels, loss, lse, dx})) return MOE_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes, vocab_backward_workspace_bytes(T, D, V, 0))) != MOE_OK) return st;
  VocabBackward a{d_loss, d_lse, x, W, VocabTargets{labels, labels_type == MOE_I64, 0, nullptr, 0}, 1.f, loss, lse,
                  nullptr, T, D, V, static_cast<uint16_t*>(dx), static_cast<uint16_t*>(dW)};
  return cuda_status(launch_vocab_backward(a, workspace, s));
}

moe_status moe_distill_forward(const void* x, const void* W, const moe_teacher* teacher, int32_t T, int32_t D, int32_t V,
                               float* loss, float* lse, float* logits, void* workspace, size_t workspace_bytes,
                               void* stream) {
  moe_status st = check_head(T, D, V);
  if (st != MOE_OK) return st;
  if ((st = check_teacher(teacher, T)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!all_there({x, W, loss, lse, logits}) || !all_on_16({x, W, loss, lse, logits})) return MOE_ERR_INVALID_ARG;
  const size_t needed = vocab_forward_workspace_bytes(T, D, V, teacher->K);
  if ((st = check_workspace(workspace, workspace_bytes, needed)) != MOE_OK) return st;
  VocabForward a{x, W, targets_of(*teacher), teacher->temperature, T, D, V, loss, lse, logits};
  return cuda_status(launch_vocab_forward(a, workspace, static_cast<cudaStream_t>(stream)));
}

moe_status moe_distill_backward(const float* d_loss, const void* x, const void* W, const moe_teacher* teacher,
                                const float* lse, const float* logits, int32_t T, int32_t D, int32_t V, void* dx,
                                void* dW, void* workspace, size_t workspace_bytes, void* stream) {
  moe_status st = check_head(T, D, V);
  if (st != MOE_OK) return st;
  if ((st = check_teacher(teacher, T)) != MOE_OK) return st;
  if (!dW || !on(dW, 16)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) return zero_weight_gradient(dW, V, D, s);
  if (!all_there({d_loss, x, W, lse, logits, dx})) return MOE_ERR_INVALID_ARG;
  if (!all_on_16({d_loss, x, W, lse, logits, dx})) return MOE_ERR_INVALID_ARG;
  const size_t needed = vocab_backward_workspace_bytes(T, D, V, teacher->K);
  if ((st = check_workspace(workspace, workspace_bytes, needed)) != MOE_OK) return st;
  VocabBackward a{d_loss, nullptr, x, W, targets_of(*teacher), teacher->temperature, nullptr, lse, logits,
                  T, D, V, static_cast<uint16_t*>(dx), static_cast<uint16_t*>(dW)};
  return cuda_status(launch_vocab_backward(a, workspace, s));
}

}  // extern "C"
