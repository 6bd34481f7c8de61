/*
 * moe_ffn.h -- C ABI of the GB300 (sm_103a) mixture-of-experts SwiGLU FFN
 * forward and backward passes, and of the operators around the layer in a
 * training step: layer norm, Newton-Schulz orthogonalisation, Muon step, and
 * the two ends of a language model: embedding, and the vocabulary product under
 * a cross entropy or a distillation loss.
 *
 * The layer (per token t of x [T, D]):
 *   logits = x[t] . Wg (+ router_bias)                 router GEMM
 *   ids[t, 0..k-1] = the k largest logits, descending,  top-k
 *                    equal logits -> lower expert index
 *   w[t, j] = softmax over the k selected logits        gate weights
 *   slots s = t*k + j are sorted stably by expert id    permutation
 *   h = silu(x W1[e]) * (x W3[e])  per routed slot      grouped GEMM W1||W3
 *   y = h W2[e]                                         grouped GEMM W2
 *   out[t] = sum_j w[t, j] * y[t, j]  (+ shared(x[t]))  weighted combine
 * Sources: "Chinchilla scaling, MoE, and fused Triton kernels", section
 * "PyTorch MoE implementation" (router, top-k, softmax over the selected
 * logits, stable argsort, bincount, grouped GEMMs, inverse permutation,
 * weighted sum); "Triton MoE Kernels & Memory Checkpointing", Part A,
 * section 2 (SwiGLU expert W2(silu(W1 x) * W3 x), top-2 of 8 routed experts
 * plus an always-on shared expert) and section 10.3 (sort-by-expert layout,
 * per-expert counts and offsets).
 *
 * Conventions for every entry point:
 *  - Pointers named *_host are host memory; every other pointer is device
 *    memory on the current CUDA device.  The caller owns all memory and the
 *    stream; the library never allocates, frees or synchronises (except
 *    moe_device_error, which reads one word back).
 *  - Tensors are contiguous and row-major.  bf16 tensors are passed as
 *    void*.  Every device pointer must be 16-byte aligned.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream).  Work is
 *    only enqueued; results are ready when the stream reaches that point.
 *  - Arguments are validated on the host before anything is enqueued.  A
 *    bad argument returns MOE_ERR_INVALID_ARG, a shape outside the limits
 *    below returns MOE_ERR_UNSUPPORTED_SHAPE; nothing is launched in either
 *    case.  A failed launch returns MOE_ERR_CUDA.  There is no fallback path.
 *  - Kernels that wait on on-chip barriers give up after a bounded time and
 *    record MOE_ERR_DEVICE_TIMEOUT in a device word, read by
 *    moe_device_error().
 *
 * Shape limits: 0 <= T <= 2^24; D and F multiples of 64 in [64, 8192]
 * (the 8192 cap is the page's hard cap on d_model and d_ff);
 * 1 <= E <= 128; 1 <= k <= min(E, 16).
 */
#ifndef MOE_FFN_H
#define MOE_FFN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,
  MOE_ERR_UNSUPPORTED_SHAPE = -2,
  MOE_ERR_CUDA = -3,
  MOE_ERR_WORKSPACE = -4,
  MOE_ERR_DEVICE_TIMEOUT = -5
} moe_status;

#define MOE_MAX_EXPERTS 128
#define MOE_MAX_TOPK 16
#define MOE_MAX_DIM 8192

/* Layer dimensions: T tokens, D = d_model, F = d_ff, E routed experts, top-k. */
typedef struct {
  int32_t T, D, F, E, k;
} moe_dims;

/* Optional per-call settings of moe_ffn_forward / moe_ffn_forward_host. */
typedef struct {
  /* cudaEvent_t handles recorded on `stream` at the stage boundaries:
   * [0] before routing, [1] after routing, [2] after the permutation,
   * [3] after W1||W3, [4] after W2, [5] after the combine.
   * moe_ffn_forward_host records [6] after the host->device copy of x (before
   * [0]) and [7] after the device->host copy of out.  moe_ffn_backward uses
   * [0..8] (see there).  NULL entries are skipped. */
  void* stage_events[12];
  /* Routing fixed from outside: ids [T, k] int32 and weights [T, k] fp32 in
   * device memory replace the router when both are non-NULL. */
  const int32_t* ids_in;
  const float* weights_in;
  /* MOE_FFN_CHAINED: run W1||W3 and W2 as one chained kernel that keeps h on
   * chip (moe_grouped_ffn_chained); needs D <= MOE_CHAINED_MAX_D.  The h
   * region of the workspace is then left untouched, and stage_events[3] is
   * recorded together with [4] after the chained kernel. */
  uint32_t flags;
} moe_ffn_options;

#define MOE_FFN_CHAINED 1u
#define MOE_CHAINED_MAX_D 256

/* Bytes of device workspace moe_ffn_forward needs for these dimensions
 * (has_shared != 0 when the shared expert is used; host_io != 0 adds the
 * device staging buffers used by moe_ffn_forward_host).  The workspace holds,
 * each 256-byte aligned: the packed router weights (moe_route_scratch_size
 * bytes), ids [T,k] i32, w [T,k] f32, block histogram
 * [ceil(T/16), E] i32 (of which the first ceil(T/TB) rows are used, TB =
 * moe_route_block_tokens(T)), counts [E] i32, offsets [E+1] i32, perm [T*k] i32,
 * inv [T*k] i32, x_sorted [T*k, D] bf16, h [T*k (+T), F] bf16,
 * y [T*k, D] bf16, (shared) ys [T, D] fp32, then (host_io) x [T, D] and
 * out [T, D] bf16. */
size_t moe_ffn_workspace_size(moe_dims d, int has_shared, int host_io);

/* Forward pass of one MoE SwiGLU FFN layer.
 *   x [T, D] bf16; Wg [D, E] bf16; router_bias [E] fp32 or NULL (added to the
 *   logits in fp32); W1, W3 [E, D, F] bf16; W2 [E, F, D] bf16;
 *   Ws1, Ws3 [D, F] and Ws2 [F, D] bf16: the shared expert, all three NULL
 *   for none; out [T, D] bf16.  Router logits and gate weights are fp32, GEMMs
 *   accumulate in fp32, h and y are stored as bf16, the combine sums in fp32
 *   and rounds once to bf16.  `workspace` holds moe_ffn_workspace_size(d,
 *   has_shared, 0) bytes; after the call it contains the routing, the
 *   permutation and the intermediates in the layout described above.
 *   opts may be NULL. */
moe_status moe_ffn_forward(const void* x, const void* Wg, const float* router_bias,
                           const void* W1, const void* W3, const void* W2,
                           const void* Ws1, const void* Ws3, const void* Ws2,
                           moe_dims d, void* out, void* workspace, size_t ws_bytes,
                           const moe_ffn_options* opts, void* stream);

/* The same forward pass with the activations in host memory: x_host [T, D]
 * bf16 is copied to the device, the layer runs, and out_host [T, D] bf16 is
 * copied back, all enqueued on `stream` (use pinned host memory for
 * asynchronous copies).  Weights stay in device memory.  `workspace` holds
 * moe_ffn_workspace_size(d, has_shared, 1) bytes. */
moe_status moe_ffn_forward_host(const void* x_host, const void* Wg, const float* router_bias,
                                const void* W1, const void* W3, const void* W2,
                                const void* Ws1, const void* Ws3, const void* Ws2,
                                moe_dims d, void* out_host, void* workspace, size_t ws_bytes,
                                const moe_ffn_options* opts, void* stream);

/* ---- Backward pass ---------------------------------------------------- */

/* Bytes of device workspace moe_ffn_backward needs.  With S_pad =
 * T*k + 64*E and R = S_pad (+T with the shared expert) it holds, each
 * 256-byte aligned: y_bar [S_pad, D], h_bar [R, F], g_bar|u_bar [R, 2F],
 * h [R, F], x_bar [R, D] (bf16, the routed rows of each expert padded to a
 * multiple of 64 rows in expert order, the shared rows from S_pad), the
 * gate-weight and selected-logit gradients [T, k] fp32, the router-
 * gradient partials ((T*k/64 + E) * (D + 1) fp32), Wg^T [E, D] bf16 and
 * the weight-gradient partial sums of groups split along their rows
 * ((kb / 80 + 2) * 2 * D * F fp32, kb = (T*k + 64 E) / 64 (+ ceil(T / 64))).
 * 0 for unsupported dimensions. */
size_t moe_ffn_backward_workspace_size(moe_dims d, int has_shared);

/* Gradients of L = sum(d_out * out) for the layer moe_ffn_forward computed
 * ("Triton MoE Kernels & Memory Checkpointing", Part A, section 8: the
 * SwiGLU expert's gradients -- h_bar split into g_bar = h_bar*u*silu'(g) and
 * u_bar = h_bar*silu(g), x_bar = g_bar W1^T + u_bar W3^T, the weight
 * gradients as outer products -- written as hand-made kernels; and the chain
 * rule through the combine, softmax and router of "Chinchilla scaling, MoE,
 * and fused Triton kernels", section "PyTorch MoE implementation").
 *   Inputs: the forward's x, Wg, W1, W3, W2, Ws1..Ws2 (as moe_ffn_forward) and
 *   d_out [T, D] bf16, plus the forward's workspace (fwd_workspace,
 *   fwd_ws_bytes >= moe_ffn_workspace_size(d, has_shared, 0)) holding the
 *   routing, permutation, x_sorted and y of that forward call; it is read
 *   only.  g and u are recomputed (the activations are not stored).
 *   Outputs: dx [T, D] bf16; dW1, dW3 [E, D, F], dW2 [E, F, D] and, with the
 *   shared expert, dWs1, dWs3 [D, F], dWs2 [F, D] in fp32 (all written, zero
 *   for an expert with no tokens); dWg [D, E] and dbias [E] fp32 (each may be
 *   NULL to skip).  Top-k is piecewise constant: unselected logits get no
 *   gradient.
 *   opts (nullable): ids_in / weights_in must repeat the fixed routing the
 *   forward was given, and then the router gets no gradient (dWg, dbias and
 *   the router term of dx are zero / skipped); stage_events [0..8] are
 *   recorded before the combine backward, after it, after h_bar, after
 *   g_bar|u_bar, after x_bar, after dW1|dW3, after dW2, after dx and after
 *   the router gradient; flags: MOE_FFN_CHAINED if the forward call ran
 *   chained (its workspace then holds no h, and the backward stores the
 *   recomputed h in its own workspace), else 0 (the W2 gradient reads the
 *   forward's h).
 *   Precision: fp32 accumulation everywhere; y_bar, h_bar, g_bar, u_bar, h
 *   and x_bar are stored as bf16 between the GEMMs; dx is summed in fp32 and
 *   rounded once.  Deterministic (no atomics).  T = 0 returns MOE_OK without
 *   touching any buffer. */
moe_status moe_ffn_backward(const void* x, const void* Wg, const void* W1, const void* W3,
                            const void* W2, const void* Ws1, const void* Ws3, const void* Ws2,
                            const void* d_out, moe_dims d, const void* fwd_workspace,
                            size_t fwd_ws_bytes, void* dx, float* dWg, float* dbias, float* dW1,
                            float* dW3, float* dW2, float* dWs1, float* dWs3, float* dWs2,
                            void* workspace, size_t ws_bytes, const moe_ffn_options* opts,
                            void* stream);

/* ---- Stage entry points (the same kernels moe_ffn_forward launches) ---- */

/* Scratch bytes moe_route needs: the router weights repacked in the MMA
 * fragment order, (D/32) * (E rounded up to 8, 16, 32, 64 or 128) * 16 bytes. */
size_t moe_route_scratch_size(moe_dims d);

/* Router GEMM + top-k + softmax ("PyTorch MoE implementation": logits, topk,
 * softmax over the selected logits).  ids [T, k] int32, weights [T, k] fp32.
 * block_hist (nullable) receives the per-block expert histogram
 * [ceil(T/TB), E] int32 over tokens [TB b, TB b + TB), TB =
 * moe_route_block_tokens(T).  scratch (device, 16-byte aligned) holds
 * moe_route_scratch_size(d) bytes. */
moe_status moe_route(const void* x, const void* Wg, const float* router_bias, moe_dims d,
                     int32_t* ids, float* weights, int32_t* block_hist, void* scratch,
                     size_t scratch_bytes, void* stream);

/* Tokens per row of the block histogram (and per block of the permutation
 * kernel) for a batch of T tokens on the current device: 64, or 32 / 16 for
 * batches too small to give each of the device's SMs two blocks; 16 when no
 * device can be queried. */
int moe_route_block_tokens(int T);

/* Scratch bytes moe_permute needs: the block histogram, sized for the most
 * rows any device uses, ceil(T/16)*E int32. */
size_t moe_permute_scratch_size(moe_dims d);

/* Stable permutation of the T*k slots by expert id (section "PyTorch MoE
 * implementation": flatten, stable argsort, bincount; "Triton MoE Kernels",
 * section 10.3, step 2: gather to expert-sorted order, counts and offsets).
 *   ids [T, k] int32 in [0, E); counts [E]; offsets [E+1] (offsets[E] = T*k);
 *   perm [T*k]: sorted position -> slot; inv [T*k]: slot -> sorted position;
 *   x [T, D] bf16 and x_sorted [T*k, D] bf16 are both NULL or both set
 *   (x_sorted[p] = x[perm[p] / k]).  Ids outside [0, E) give undefined
 *   output.  scratch holds moe_permute_scratch_size(d) bytes. */
moe_status moe_permute(const int32_t* ids, moe_dims d, int32_t* counts, int32_t* offsets,
                       int32_t* perm, int32_t* inv, const void* x, void* x_sorted,
                       void* scratch, size_t scratch_bytes, void* stream);

/* Grouped GEMM W1||W3 with the SwiGLU epilogue ("Triton MoE Kernels",
 * sections 2 and 10.2): for each expert e and sorted row p in
 * [offsets[e], offsets[e+1]): h[p] = silu(x_sorted[p] W1[e]) * (x_sorted[p] W3[e]).
 * With the shared expert (Ws1, Ws3 non-NULL, x non-NULL) rows T*k + t of h
 * receive silu(x[t] Ws1) * (x[t] Ws3).  h holds T*k (+T) rows of F bf16. */
moe_status moe_grouped_swiglu(const void* x_sorted, const void* x, const void* W1, const void* W3,
                              const void* Ws1, const void* Ws3, const int32_t* offsets,
                              moe_dims d, void* h, void* stream);

/* Grouped GEMM W2: y[p] = h[p] W2[e] for the routed rows, y [T*k, D] bf16;
 * with the shared expert (Ws2 non-NULL) also ys[t] = h[T*k + t] Ws2, ys
 * [T, D] fp32 (required then, ignored otherwise).  The shared expert's output
 * is added to the layer's output with weight 1, so it keeps its fp32
 * accumulation instead of being rounded to bf16 first. */
moe_status moe_grouped_down(const void* h, const void* W2, const void* Ws2, const int32_t* offsets,
                            moe_dims d, void* y, float* ys, void* stream);

/* W1||W3 + SiLU*mul and W2 chained in one kernel, h never written to memory
 * ("Chinchilla scaling, MoE, and fused Triton kernels", sections "Fused Triton
 * kernel mechanism" and "Triton fused kernel implementation").  Same inputs as
 * moe_grouped_swiglu and moe_grouped_down together, same outputs y [T*k, D]
 * bf16 and (shared) ys [T, D] fp32: per 256-row tile the kernel streams F in
 * 64-column chunks, rounds each h chunk to bf16 in shared memory and
 * accumulates y in fp32 over the chunks in the order of the two separate
 * GEMMs, so y and ys equal their result.
 * MOE_ERR_UNSUPPORTED_SHAPE when D > MOE_CHAINED_MAX_D: a tile's y
 * accumulator (D fp32 columns per row) and two g|u buffers (128 columns each)
 * must fit in the 512 TMEM columns of an SM. */
moe_status moe_grouped_ffn_chained(const void* x_sorted, const void* x, const void* W1,
                                   const void* W3, const void* W2, const void* Ws1,
                                   const void* Ws3, const void* Ws2, const int32_t* offsets,
                                   moe_dims d, void* y, float* ys, void* stream);

/* Weighted combine ("PyTorch MoE implementation": inverse permutation and
 * weighted sum): out[t] = sum_j weights[t, j] * y[inv[t*k + j]] (+ ys[t] when
 * ys, the shared expert's rows [T, D] fp32, is non-NULL), summed in fp32 in
 * order j = 0..k-1 and then the shared term, rounded once to bf16. */
moe_status moe_combine(const void* y, const float* ys, const float* weights, const int32_t* inv, moe_dims d,
                       void* out, void* stream);

/* ---- Layer norm around the layer ---- */

/* Element types of the entry points below that take more than one. */
typedef enum { MOE_BF16 = 0, MOE_FP32 = 1 } moe_dtype;

/* Layer norm of the residual stream, with the sum it starts from:
 *   h = x (+ add), rounded once to x's type when `add` is given
 *   y = (h - mean(h)) * rstd * weight (+ bias),  rstd = 1/sqrt(var(h) + eps)
 * per row of D elements; mean and var (the mean squared distance from the
 * mean) are fp32 sums over the h that is stored.
 *   x [T, D] of type x_type; add [T, D] bf16 or NULL; weight, bias [D] fp32
 *   (bias may be NULL); y [T, D] bf16; h [T, D] of x's type, exactly when
 *   `add` is given (else NULL); mean, rstd [T] fp32.
 * 1 <= D <= 8192, any D; 0 <= T <= 2^24; eps >= 0 and finite.  h may be x
 * itself; no other output may overlap an input. */
moe_status moe_layer_norm_forward(const void* x, moe_dtype x_type, const void* add, const float* weight,
                                  const float* bias, float eps, int32_t T, int32_t D, void* y, void* h,
                                  float* mean, float* rstd, void* stream);

/* Bytes of scratch moe_layer_norm_backward needs (0 for a bad shape). */
size_t moe_layer_norm_backward_scratch_size(int32_t T, int32_t D);

/* Gradients of sum(dy * y) (+ sum(d_stream * h)) for the forward above:
 *   n = (x - mean) * rstd, p = dy * weight,
 *   dx = rstd * (p - mean(p) - n * mean(p * n)) (+ d_stream)
 *   dweight = sum_t dy * n,  dbias = sum_t dy
 *   dy [T, D] bf16; x [T, D] of type x_type: the rows that were normalised
 *   (h where the forward added); d_stream [T, D] of x's type or NULL: the
 *   gradient that reaches the same rows past the norm; dx [T, D] of x's type;
 *   dweight [D], dbias [D] fp32 (dbias may be NULL).  dx may be d_stream
 *   itself.  The sums over tokens run in a fixed order (the same bits every
 *   time on one device).  T = 0 writes zero weight gradients. */
moe_status moe_layer_norm_backward(const void* dy, const void* x, moe_dtype x_type, const float* weight,
                                   const float* mean, const float* rstd, const void* d_stream, int32_t T,
                                   int32_t D, void* dx, float* dweight, float* dbias, void* scratch,
                                   size_t scratch_bytes, void* stream);

/* ---- Orthogonalised updates of the expert matrices ---- */

#define MOE_MAX_STACKS 16    /* stacks in one moe_muon_step call */
#define MOE_MAX_NS_STEPS 16  /* Newton-Schulz steps */
#define MOE_MAX_MATRICES 4096 /* matrices in one call */

/* Bytes of device workspace for `count` matrices of rows x cols (or of
 * cols x rows); 0 for a bad shape. */
size_t moe_newton_schulz_workspace_size(int32_t count, int32_t rows, int32_t cols);

/* Newton-Schulz orthogonalisation of each of `count` matrices G [rows, cols]:
 *   X = G / (|G|_F + eps)
 *   steps times, with the step's (a, b, c):
 *     A = X X^T;  X <- a X + (b A + c A A) X     (X^T X where rows > cols)
 *   grad [count, rows, cols] of type grad_type; out [count, rows, cols] bf16;
 *   coefficients: steps x 3 floats in host memory, read before the call
 *   returns.  The products take fp16 operands and fp32 sums, the linear term
 *   keeps X to about 14 bits (to fp32 where the short side is at most 128 and
 *   the long one at most 2048; such matrices stay on chip and leave the
 *   workspace untouched).  Before its rounding to bf16, which is 1.7e-3, the
 *   result is 0.6e-3 to 1.6e-3 off in the 2-norm (2.1e-3 at 16 rows); no option
 *   takes more bits.  The coefficients have to keep the singular values of X
 *   below 5 (those in common use keep them below 1.3).  A matrix with an element
 *   that is no finite number, or with a sum of squares past fp32, becomes NaN;
 *   the others of the stack do not.  At the other end, |G|_F under 1e-20 counts
 *   as 0 beside eps (which then has to be more than 0), and off the chip
 *   elements of X under 7e-12, as |G|_F far below eps leaves them, become 0.
 * 1 <= rows, cols <= 8192; 0 <= count <= MOE_MAX_MATRICES;
 * 1 <= steps <= MOE_MAX_NS_STEPS. */
moe_status moe_newton_schulz(const void* grad, moe_dtype grad_type, int32_t count, int32_t rows, int32_t cols,
                             int32_t steps, const float* coefficients, float eps, void* out, void* workspace,
                             size_t workspace_bytes, void* stream);

/* One stack of weight matrices of moe_muon_step. */
typedef struct {
  void* weight;        /* [count, rows, cols], updated in place */
  const void* grad;    /* [count, rows, cols] */
  float* momentum;     /* [count, rows, cols] fp32, updated in place */
  void* weight_bf16;   /* with fp32 weights: [count, rows, cols] bf16, written
                        * with the updated weights; or NULL */
  int32_t count, rows, cols;
} moe_matrix_stack;

typedef struct {
  float lr, momentum, weight_decay, scale, eps;
  int32_t nesterov;           /* 0 or 1 */
  int32_t steps;
  const float* coefficients;  /* steps x 3, host memory */
} moe_muon_params;

/* One Muon step on n_stacks stacks of matrices, all of the same shape up to
 * transposition (W1, W3 [E, D, F] and W2 [E, F, D] of a layer go together):
 *   m <- momentum m + g;  u = g + momentum m (nesterov) or m
 *   w <- (1 - lr weight_decay) w - lr scale NS(u)
 * with NS as in moe_newton_schulz.  `stacks` is host memory, read before the
 * call returns.  The workspace is that of the stacks' total count. */
moe_status moe_muon_step(const moe_matrix_stack* stacks, int32_t n_stacks, moe_dtype grad_type,
                         moe_dtype weight_type, const moe_muon_params* params, void* workspace,
                         size_t workspace_bytes, void* stream);

/* ---- The ends of a language model: embedding, loss over the vocabulary ---- */

#define MOE_MAX_VOCAB (1 << 22) /* rows of a table */
#define MOE_MAX_TEACHER 256     /* teacher entries a token */

typedef enum { MOE_I32 = 0, MOE_I64 = 1 } moe_index_type;

/* Embedding lookup:  out[t] = scale * table[ids[t]], rounded once.
 *   ids [T] of type ids_type; an id outside [0, V) gives a row of zeros;
 *   table [V, D] of type table_type; out [T, D] of type out_type.
 * 1 <= D <= 8192, any D; 1 <= V <= MOE_MAX_VOCAB; 0 <= T <= 2^24; scale finite.
 * Here and below no output may overlap an input. */
moe_status moe_embedding_forward(const void* ids, moe_index_type ids_type, const void* table,
                                 moe_dtype table_type, float scale, int32_t T, int32_t V, int32_t D,
                                 void* out, moe_dtype out_type, void* stream);

/* Bytes of scratch moe_embedding_backward needs (0 for a bad shape). */
size_t moe_embedding_backward_scratch_size(int32_t T, int32_t V, int32_t D);

/* Gradient of sum(d_out * out) for the forward above:
 *   d_table[v] = (add[v] +) scale * sum over t with ids[t] = v of d_out[t]
 *   d_out [T, D] of type d_type; add [V, D] bf16 or NULL: a gradient that
 *   reaches the table elsewhere (the dW of the calls below, where the table is
 *   the head's too); d_table [V, D] fp32.  The tokens are sorted, and the sums
 *   run in fp32 in a fixed order (the same bits every time). */
moe_status moe_embedding_backward(const void* d_out, moe_dtype d_type, const void* ids,
                                  moe_index_type ids_type, float scale, const void* add, int32_t T,
                                  int32_t V, int32_t D, float* d_table, void* scratch,
                                  size_t scratch_bytes, void* stream);

/* Limits of the four calls below: 1 <= T <= 2^24 (T = 0 does nothing, or gives
 * zero weight gradients); D a multiple of 64 in [64, 8192]; 1 <= V <= MOE_MAX_VOCAB.
 * x [T, D] and the table W [V, D] are bf16.  z = x W^T has fp32 sums and never
 * reaches memory: the tensor cores sum up to 896 products, cutting to 24 bits at
 * each step, and these sums are added in fp32.  Products of one sign leave z up to
 * 2e-6 of itself too near to 0, others less than 1e-6 of the size of their sums;
 * where 24 bits hold every sum, z is exact.  Workspaces start on 256 bytes and
 * hold nothing between calls; the size functions return 0 for a bad shape.
 * n_teacher is 0 for the cross entropy.  The forward's is a float pair or so a
 * token and 256 to 1024 words.  The backward's holds the logits' gradient of a
 * piece of the vocabulary in bf16, 2 T V bytes but at most the larger of 4 GiB and
 * 4096 T (2048 words, 64 GiB at T = 2^24), and fp32 sums of dx and dW where their
 * reductions are cut. */
size_t moe_vocab_forward_workspace_size(int32_t T, int32_t D, int32_t V, int32_t n_teacher);
size_t moe_vocab_backward_workspace_size(int32_t T, int32_t D, int32_t V, int32_t n_teacher);

/* Softmax cross entropy over the vocabulary:
 *   lse[t] = log sum_v exp(z[t, v]),  loss[t] = lse[t] - z[t, labels[t]]
 * A label outside [0, V) is a token without a loss: loss 0 (lse as above). */
moe_status moe_cross_entropy_forward(const void* x, const void* W, const void* labels,
                                     moe_index_type labels_type, int32_t T, int32_t D, int32_t V,
                                     float* loss, float* lse, void* workspace, size_t workspace_bytes,
                                     void* stream);

/* Gradients of sum(d_loss * loss) (+ sum(d_lse * lse)) for the call above:
 *   dz[t, v] = d_loss[t] (exp(z[t, v] - lse[t]) - [v = labels[t]])
 *              + d_lse[t] exp(z[t, v] - lse[t])
 *   dx = dz W [T, D] bf16,  dW = dz^T x [V, D] bf16
 * d_loss [T] fp32 (not read where a token has no loss); d_lse [T] fp32 or
 * NULL; loss and lse: the forward's.  z is computed again, piece by piece of
 * the vocabulary; dz is rounded to bf16 for its two products, whose sums are
 * fp32.  A token with neither gradient has dx = 0 whatever its x holds, but dW
 * takes 0 x, so x has to be finite. */
moe_status moe_cross_entropy_backward(const float* d_loss, const float* d_lse, const void* x,
                                      const void* W, const void* labels, moe_index_type labels_type,
                                      const float* loss, const float* lse, int32_t T, int32_t D,
                                      int32_t V, void* dx, void* dW, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* A teacher's top logits for each token. */
typedef struct {
  const void* ids;       /* [T, K] of type ids_type; outside [0, V): no entry */
  const void* logits;    /* [T, K] of type logits_type; -inf: no entry */
  moe_index_type ids_type;
  moe_dtype logits_type;
  int32_t K;             /* 1 <= K <= MOE_MAX_TEACHER */
  float temperature;     /* > 0, finite, and so that 2 / temperature is */
} moe_teacher;

/* Distillation from the teacher's entries, with p = softmax of its logits over
 * temperature among the token's entries:
 *   lse[t] = log sum_v exp(z[t, v] / temperature)
 *   loss[t] = sum_j p[t, j] (log p[t, j] - z[t, ids[t, j]] / temperature + lse[t])
 * loss, lse [T] fp32; logits [T, K] fp32: z at the ids (0 where there is no
 * entry for the id's sake).  A token without entries has loss 0; an id that
 * comes twice counts twice. */
moe_status moe_distill_forward(const void* x, const void* W, const moe_teacher* teacher, int32_t T,
                               int32_t D, int32_t V, float* loss, float* lse, float* logits,
                               void* workspace, size_t workspace_bytes, void* stream);

/* Gradients of sum(d_loss * loss) for the call above, as in
 * moe_cross_entropy_backward:
 *   dz[t, v] = d_loss[t] / temperature (exp(z[t, v] / temperature - lse[t])
 *              - sum over j with ids[t, j] = v of p[t, j])
 * lse, logits: the forward's. */
moe_status moe_distill_backward(const float* d_loss, const void* x, const void* W,
                                const moe_teacher* teacher, const float* lse, const float* logits,
                                int32_t T, int32_t D, int32_t V, void* dx, void* dW, void* workspace,
                                size_t workspace_bytes, void* stream);

/* ---- Allocation-free variant ---- */

/* moe_permute without a caller-provided scratch buffer, for callers that
 * cannot allocate device memory (for example a plugin inside a host framework
 * that owns all device memory, or a path that must never call cudaMalloc).
 * The pages have no counterpart of this entry point; it exists for such
 * callers only.  Arguments and results are those of moe_permute.  The block
 * histogram lives in a fixed 65,536-entry int32 array (256 KB) in the
 * library's own device memory, held on every GPU that loads the library until
 * the process exits; calls with ceil(T/TB) * E > 65,536 (TB =
 * moe_route_block_tokens(T)) return
 * MOE_ERR_UNSUPPORTED_SHAPE.  Every call shares that array: calls whose work
 * overlaps on the GPU race and must be serialised by the caller.  The first
 * call on each device looks up the array's device address (with that device
 * current); make it before any stream capture.  It calls no cudaMalloc or
 * cudaFree. */
moe_status moe_permute_noalloc(const int32_t* ids, moe_dims d, int32_t* counts, int32_t* offsets,
                               int32_t* perm, int32_t* inv, const void* x, void* x_sorted,
                               void* stream);

/* ---- Diagnostics ---- */

/* Reads and clears the device error word of the current device (a
 * synchronous copy).  Returns MOE_OK or MOE_ERR_DEVICE_TIMEOUT. */
moe_status moe_device_error(void);

/* Failure-detection self-test: launches one CTA whose bounded mbarrier wait
 * (the wait every pipelined kernel of the library uses) can never complete;
 * it gives up after timeout_us (1 .. 10^6 microseconds), writes 1 to
 * *gave_up (device int32) and records the timeout, so that a following
 * moe_device_error() returns MOE_ERR_DEVICE_TIMEOUT.  The GPU context stays
 * usable: nothing faults and nothing is left running. */
moe_status moe_selftest_wait_timeout(int timeout_us, int32_t* gave_up, void* stream);

/* moe_embedding_backward as it runs on a device that holds no thread-block
 * cluster of 16: 4097 to 65536 tokens are sorted by a launch a pass, not on chip.
 * The result has the same bits. */
moe_status moe_selftest_embedding_by_passes(const void* d_out, moe_dtype d_type, const void* ids,
                                            moe_index_type ids_type, float scale, const void* add, int32_t T,
                                            int32_t V, int32_t D, float* d_table, void* scratch,
                                            size_t scratch_bytes, void* stream);

/* Number of kernels this library has launched since it was loaded. */
uint64_t moe_launch_count(void);

/* Static text for a status code. */
const char* moe_status_str(moe_status s);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FFN_H */
