// Layer norm of the residual stream in front of the MoE FFN, and its backward
// pass.
//
//   forward   h = x (+ add), mu = mean(h), v = mean((h - mu)^2),
//             r = 1 / sqrt(v + eps), y = (h - mu) r w (+ b)
//   backward  n = (x - mu) r, p = dy w,
//             dx = r (p - mean(p) - n mean(p n)) (+ d_stream),
//             dw = sum_t dy n, db = sum_t dy
//
// A row is held in registers by P threads (a warp up to 1024 columns), so it
// is read once and the variance is the sum of squared distances from the mean
// and not a difference of two large sums.  All sums are fp32.  The weight
// gradients are summed in two stages in a fixed order: every block adds its
// rows in registers and writes one partial row, and a second kernel adds the
// partial rows; there are no atomics, so the results do not change from run
// to run.
#include "moe_device.cuh"
#include "moe_kernels.cuh"

namespace moe {

namespace {

constexpr int kLnThreads = 256;
constexpr int kLnWarps = kLnThreads / 32;

// VEC consecutive elements as floats; p is aligned to VEC elements.
template <int VEC>
MOE_DEV void load_vec(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = __ldcs(p);
  }
}

template <int VEC>
MOE_DEV void load_vec(const uint16_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(u[i]), v[2 * i + 1] = bf16_hi(u[i]);
  } else {
    v[0] = bf16_lo(__ldcs(p));
  }
}

// Weights: re-read for every row, so through the L1 cache.
template <int VEC>
MOE_DEV void load_weight(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = __ldg(p);
  }
}

template <int VEC>
MOE_DEV void store_vec(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    p[0] = v[0];
  }
}

template <int VEC>
MOE_DEV void store_vec(uint16_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    p[0] = static_cast<uint16_t>(pack_bf16x2(v[0], 0.f));
  }
}

// The value as the stream's type holds it.
MOE_DEV float as_stored(float v, const float*) { return v; }
MOE_DEV float as_stored(float v, const uint16_t*) { return bf16_lo(pack_bf16x2(v, 0.f)); }

// Sums over the P threads of a row; `red` is only used when P spans warps.
// Every thread of the block calls it.
template <int P>
MOE_DEV float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (P > 32) {
    const int warp = threadIdx.x >> 5;
    constexpr int kPerRow = P / 32;
    __syncthreads();  // the previous sum has been read
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const int first = warp / kPerRow * kPerRow;
    v = red[first];
#pragma unroll
    for (int i = 1; i < kPerRow; ++i) v += red[first + i];
  }
  return v;
}

template <typename XT, int P, int N, int VEC, bool ADD>
__global__ void __launch_bounds__(kLnThreads) layer_norm_kernel(
    const XT* __restrict__ x, const uint16_t* __restrict__ add, const float* __restrict__ w,
    const float* __restrict__ b, float eps, int T, int D, uint16_t* __restrict__ y, XT* __restrict__ h,
    float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[kLnWarps];
  constexpr int kRows = kLnThreads / P;
  const int t = threadIdx.x % P;
  const int row = blockIdx.x * kRows + threadIdx.x / P;
  const bool live = row < T;
  const size_t base = static_cast<size_t>(live ? row : 0) * D;
  float v[N][VEC];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * P + t) * VEC;
    if (live && c < D) {
      load_vec<VEC>(x + base + c, v[i]);
      if constexpr (ADD) {
        float a[VEC];
        load_vec<VEC>(add + base + c, a);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] = as_stored(v[i][j] + a[j], x);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += v[i][j];
    }
  }
  const float inv_d = 1.f / static_cast<float>(D);
  const float mu = row_sum<P>(s, red) * inv_d;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * P + t) * VEC;
    if (live && c < D) {
      if constexpr (ADD) store_vec<VEC>(h + base + c, v[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] -= mu;
        q = fmaf(v[i][j], v[i][j], q);
      }
    }
  }
  const float r = 1.f / sqrtf(row_sum<P>(q, red) * inv_d + eps);
  if (!live) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * P + t) * VEC;
    if (c < D) {
      float wv[VEC], o[VEC];
      load_weight<VEC>(w + c, wv);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = v[i][j] * r * wv[j];
      if (b != nullptr) {
        load_weight<VEC>(b + c, wv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] += wv[j];
      }
      store_vec<VEC>(y + base + c, o);
    }
  }
  if (t == 0) {
    mean[row] = mu;
    rstd[row] = r;
  }
}

// Backward: block k takes row groups k, k + gridDim.x, ...; part[k] = its
// sums of dy n (first D) and dy (next D).
template <typename XT, int P, int N, int VEC, bool STREAM>
__global__ void __launch_bounds__(kLnThreads) layer_norm_bwd_kernel(
    const uint16_t* __restrict__ dy, const XT* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ mean, const float* __restrict__ rstd, const XT* __restrict__ d_stream, int T, int D,
    XT* __restrict__ dx, float* __restrict__ part) {
  extern __shared__ float acc[];  // [2][D]
  __shared__ float red[2 * kLnWarps];
  constexpr int kRows = kLnThreads / P;
  const int t = threadIdx.x % P, group = threadIdx.x / P;
  float dw[N][VEC], db[N][VEC];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.f;
  const float inv_d = 1.f / static_cast<float>(D);
  // every thread of the block makes the same number of turns: row_sum has barriers
  for (int row0 = blockIdx.x * kRows; row0 < T; row0 += gridDim.x * kRows) {
    const int row = row0 + group;
    const bool live = row < T;
    const size_t base = static_cast<size_t>(live ? row : 0) * D;
    const float mu = live ? mean[row] : 0.f, r = live ? rstd[row] : 0.f;
    float n[N][VEC], p[N][VEC];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * P + t) * VEC;
      if (live && c < D) {
        float wv[VEC];
        load_vec<VEC>(x + base + c, n[i]);
        load_vec<VEC>(dy + base + c, p[i]);
        load_weight<VEC>(w + c, wv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          n[i][j] = (n[i][j] - mu) * r;
          dw[i][j] = fmaf(p[i][j], n[i][j], dw[i][j]);
          db[i][j] += p[i][j];
          p[i][j] *= wv[j];
          s1 += p[i][j];
          s2 = fmaf(p[i][j], n[i][j], s2);
        }
      }
    }
    const float c1 = row_sum<P>(s1, red) * inv_d;
    const float c2 = row_sum<P>(s2, red + kLnWarps) * inv_d;
    if (live) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * P + t) * VEC;
        if (c < D) {
          float o[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) o[j] = r * (p[i][j] - c1 - n[i][j] * c2);
          if constexpr (STREAM) {
            float g[VEC];
            load_vec<VEC>(d_stream + base + c, g);
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] += g[j];
          }
          store_vec<VEC>(dx + base + c, o);
        }
      }
    }
  }
  // the block's row groups add their columns one after the other
  for (int g = 0; g < kRows; ++g) {
    if (group == g) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * P + t) * VEC;
        if (c < D) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            acc[c + j] = g == 0 ? dw[i][j] : acc[c + j] + dw[i][j];
            acc[D + c + j] = g == 0 ? db[i][j] : acc[D + c + j] + db[i][j];
          }
        }
      }
    }
    __syncthreads();
  }
  float* out = part + static_cast<size_t>(blockIdx.x) * 2 * D;
  for (int c = threadIdx.x; c < 2 * D; c += kLnThreads) out[c] = acc[c];
  griddep_launch_dependents();
}

// out[c] = sum over the nblk partial rows, column c of [2 D]: 32 columns a
// block, 8 strips of rows added in order.
__global__ void __launch_bounds__(256) layer_norm_reduce_kernel(const float* __restrict__ part, int nblk, int D,
                                                                float* __restrict__ dweight,
                                                                float* __restrict__ dbias) {
  __shared__ float strip[8][32];
  griddep_wait();  // the partial rows come from the previous kernel
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * D)
    for (int i = k; i < nblk; i += 8) s += part[static_cast<size_t>(i) * 2 * D + c];
  strip[k][lane] = s;
  __syncthreads();
  if (k == 0 && c < 2 * D) {
    s = strip[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) s += strip[i][lane];
    if (c < D)
      dweight[c] = s;
    else if (dbias != nullptr)
      dbias[c - D] = s;
  }
}

template <typename XT, int P, int N, int VEC>
cudaError_t run_fwd(const LayerNormArgs& a, cudaStream_t s) {
  constexpr int kRows = kLnThreads / P;
  const dim3 grid((a.T + kRows - 1) / kRows);
  auto kernel = a.add ? layer_norm_kernel<XT, P, N, VEC, true> : layer_norm_kernel<XT, P, N, VEC, false>;
  return launch_kernel(kernel, grid, dim3(kLnThreads), 0, s, false, static_cast<const XT*>(a.x),
                       static_cast<const uint16_t*>(a.add), a.weight, a.bias, a.eps, a.T, a.D,
                       static_cast<uint16_t*>(a.y), static_cast<XT*>(a.h), a.mean, a.rstd);
}

template <typename XT, int P, int N, int VEC>
cudaError_t run_bwd(const LayerNormBwdArgs& a, cudaStream_t s) {
  constexpr int kRows = kLnThreads / P;
  const int sms = current_device_sms();
  int nblk = (a.T + kRows - 1) / kRows;
  if (nblk > 2 * sms) nblk = 2 * sms;
  if (nblk > kLnMaxPartials) nblk = kLnMaxPartials;
  auto kernel = a.d_stream ? layer_norm_bwd_kernel<XT, P, N, VEC, true> : layer_norm_bwd_kernel<XT, P, N, VEC, false>;
  const size_t smem = static_cast<size_t>(2) * a.D * sizeof(float);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if (nblk > 0)  // no rows: the sums below are zeros
    e = launch_kernel(kernel, dim3(nblk), dim3(kLnThreads), smem, s, false, static_cast<const uint16_t*>(a.dy),
                      static_cast<const XT*>(a.x), a.weight, a.mean, a.rstd, static_cast<const XT*>(a.d_stream), a.T,
                      a.D, static_cast<XT*>(a.dx), a.part);
  if (e != cudaSuccess) return e;
  return launch_kernel(layer_norm_reduce_kernel, dim3((2 * a.D + 31) / 32), dim3(256), 0, s, true,
                       static_cast<const float*>(a.part), nblk, a.D, a.dweight, a.dbias);
}

// P threads a row: 32 up to 1024 columns, then 64, 128, 256, so that a thread
// holds at most 32 values.  Rows that are no multiple of 16 bytes go element
// by element.
template <typename XT, typename Args, cudaError_t (*R32_1)(const Args&, cudaStream_t),
          cudaError_t (*R32_2)(const Args&, cudaStream_t), cudaError_t (*R32_3)(const Args&, cudaStream_t),
          cudaError_t (*R32_4)(const Args&, cudaStream_t), cudaError_t (*R64)(const Args&, cudaStream_t),
          cudaError_t (*R128)(const Args&, cudaStream_t), cudaError_t (*R256)(const Args&, cudaStream_t),
          cudaError_t (*S32)(const Args&, cudaStream_t), cudaError_t (*S64)(const Args&, cudaStream_t),
          cudaError_t (*S128)(const Args&, cudaStream_t), cudaError_t (*S256)(const Args&, cudaStream_t)>
cudaError_t dispatch(const Args& a, cudaStream_t s) {
  if (a.D % 8 == 0) {
    if (a.D <= 256) return R32_1(a, s);
    if (a.D <= 512) return R32_2(a, s);
    if (a.D <= 768) return R32_3(a, s);
    if (a.D <= 1024) return R32_4(a, s);
    if (a.D <= 2048) return R64(a, s);
    if (a.D <= 4096) return R128(a, s);
    return R256(a, s);
  }
  if (a.D <= 1024) return S32(a, s);
  if (a.D <= 2048) return S64(a, s);
  if (a.D <= 4096) return S128(a, s);
  return S256(a, s);
}

template <typename XT>
cudaError_t dispatch_fwd(const LayerNormArgs& a, cudaStream_t s) {
  return dispatch<XT, LayerNormArgs, run_fwd<XT, 32, 1, 8>, run_fwd<XT, 32, 2, 8>, run_fwd<XT, 32, 3, 8>,
                  run_fwd<XT, 32, 4, 8>, run_fwd<XT, 64, 4, 8>, run_fwd<XT, 128, 4, 8>, run_fwd<XT, 256, 4, 8>,
                  run_fwd<XT, 32, 32, 1>, run_fwd<XT, 64, 32, 1>, run_fwd<XT, 128, 32, 1>, run_fwd<XT, 256, 32, 1>>(
      a, s);
}

template <typename XT>
cudaError_t dispatch_bwd(const LayerNormBwdArgs& a, cudaStream_t s) {
  return dispatch<XT, LayerNormBwdArgs, run_bwd<XT, 32, 1, 8>, run_bwd<XT, 32, 2, 8>, run_bwd<XT, 32, 3, 8>,
                  run_bwd<XT, 32, 4, 8>, run_bwd<XT, 64, 4, 8>, run_bwd<XT, 128, 4, 8>, run_bwd<XT, 256, 4, 8>,
                  run_bwd<XT, 32, 32, 1>, run_bwd<XT, 64, 32, 1>, run_bwd<XT, 128, 32, 1>, run_bwd<XT, 256, 32, 1>>(
      a, s);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s) {
  return a.x_fp32 ? dispatch_fwd<float>(a, s) : dispatch_fwd<uint16_t>(a, s);
}

cudaError_t launch_layer_norm_bwd(const LayerNormBwdArgs& a, cudaStream_t s) {
  return a.x_fp32 ? dispatch_bwd<float>(a, s) : dispatch_bwd<uint16_t>(a, s);
}

}  // namespace moe
