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
#include <algorithm>
#include <mutex>

#include "moe_device.cuh"
#include "moe_kernels.cuh"

namespace moe {

namespace {

constexpr int kLnThreads = 256;
constexpr int kLnWarps = kLnThreads / 32;
constexpr int kLnMaxStages = 6;                   // slots of the backward's ring
constexpr size_t kLnHalfSm = 108 * 1024;          // shared memory of a block when two share an SM
constexpr size_t kLnWholeSm = 216 * 1024;

// One contiguous piece of global memory into shared memory; 16-byte aligned,
// a multiple of 16 bytes.
MOE_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

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

// Results are not read again soon: with the streaming policy the forward at T =
// 32768, D = 768 takes 33.9 us instead of 36.3.
template <int VEC>
MOE_DEV void store_vec(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
  } else {
    p[0] = v[0];
  }
}

template <int VEC>
MOE_DEV void store_vec(uint16_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
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

// Blocks an SM that the compiler keeps registers for: six for bf16 rows of up
// to 512 columns, and with a residual sum up to 768; else its own choice.
// Device time at 50 MB of x, bf16, with the bound / without: with the sum D =
// 256 33.9 / 33.9 us, 512 33.2 / 35.4, 768 33.8 / 38.7 (seven blocks: 40.2),
// 1024 37.5 / 38.4, 2048 39.5 / 41.2; without it 512 21.9 / 22.6, 768 24.7 /
// 22.1, 1024 27.9 / 22.4, 2048 28.6 / 23.9.  fp32 (100 MB): 512 45.7 / 45.7
// and 26.7 / 26.1, 768 47.8 / 47.8 and 26.2 / 25.8.
template <typename XT, int N, int VEC, bool ADD>
constexpr int kFwdBlocks = VEC == 8 && sizeof(XT) == 2 && N <= (ADD ? 3 : 2) ? 6 : 1;

// h may be x itself (no __restrict__): a thread stores only what it has loaded.
template <typename XT, int P, int N, int VEC, bool ADD>
__global__ void __launch_bounds__(kLnThreads, kFwdBlocks<XT, N, VEC, ADD>) layer_norm_kernel(
    const XT* x, const uint16_t* __restrict__ add, const float* __restrict__ w, const float* __restrict__ b, float eps,
    int T, int D, uint16_t* __restrict__ y, XT* h, float* __restrict__ mean, float* __restrict__ rstd) {
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
        store_vec<VEC>(h + base + c, v[i]);  // at once: after the sums it took 75 us instead of 64 (fp32, D = 2048)
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

// The block's row groups have left their sums side by side, [kRows][2][D]:
// adds them column by column into the block's partial row, or, when it is the
// only block, into the results.
template <int kRows>
MOE_DEV void block_sums(const float* sums, int D, float* part, float* dweight, float* dbias) {
  __syncthreads();
  float* out = part + static_cast<size_t>(blockIdx.x) * 2 * D;
  for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) {
    float v = sums[c];
#pragma unroll
    for (int g = 1; g < kRows; ++g) v += sums[g * 2 * D + c];
    if (gridDim.x > 1)
      out[c] = v;
    else if (c < D)
      dweight[c] = v;
    else if (dbias != nullptr)
      dbias[c - D] = v;
  }
  griddep_launch_dependents();
}

// Backward: block k takes row groups k, k + gridDim.x, ...; part[k] = its
// sums of dy n (first D) and dy (next D).  This form, one element at a time,
// is for rows that are no multiple of 16 bytes.  dx may be d_stream itself (no
// __restrict__ on the two, here and below): an element is read before it is
// written, by the same thread or into the row's slot.
template <typename XT, int P, int N, bool STREAM>
__global__ void __launch_bounds__(kLnThreads) layer_norm_bwd_kernel(
    const uint16_t* __restrict__ dy, const XT* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ mean, const float* __restrict__ rstd, const XT* d_stream, int T, int D,
    XT* dx, float* __restrict__ part, float* __restrict__ dweight, float* __restrict__ dbias) {
  constexpr int VEC = 1;
  extern __shared__ float sums[];  // [kRows][2][D]
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
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = i * P + t;
    if (c < D) {
      sums[(group * 2) * D + c] = dw[i][0];
      sums[(group * 2 + 1) * D + c] = db[i][0];
    }
  }
  block_sums<kRows>(sums, D, part, dweight, dbias);
}

// Rows that are multiples of 16 bytes come through a ring in shared memory:
// each of `stages` slots holds the rows of one turn of the block (dy, x,
// d_stream, one bulk copy each), which a warp of its own asks for a few turns
// ahead, so that 100 to 200 KB are on the way on each SM without a register
// held for them.  (Loads straight into registers left DRAM at 29%, a ring of
// single rows filled by their own warps, with 1.5 KB copies, at 28%.)  A row
// is read from its slot twice, for the sums and for dx, rather than kept.
constexpr int kRingThreads = kLnThreads + 32;

template <typename XT>
__host__ __device__ constexpr int slot_bytes(int rows, int D, bool stream) {
  return rows * D * (2 + static_cast<int>(sizeof(XT)) * (stream ? 2 : 1));
}

// All P threads of a row.
template <int P>
MOE_DEV void row_sync(int group) {
  if constexpr (P == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(P) : "memory");
}

// Pairs of fp32 in one register pair: one instruction for two.
typedef unsigned long long f2;
MOE_DEV f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
MOE_DEV float2 unpack2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
MOE_DEV f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
MOE_DEV f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
MOE_DEV f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Two sums over the P threads of a row.
template <int P>
MOE_DEV void row_sum2(float& a, float& b, int group, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (P > 32) {
    constexpr int kPerRow = P / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = make_float2(a, b);
    row_sync<P>(group);
    const int first = warp / kPerRow * kPerRow;
    a = red[first].x, b = red[first].y;
#pragma unroll
    for (int i = 1; i < kPerRow; ++i) a += red[first + i].x, b += red[first + i].y;
  }
}

// Eight values of a slot (or of the weights) as four pairs.
MOE_DEV void slot_vec(const float* p, f2 (&v)[4]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = pack2(a.x, a.y), v[1] = pack2(a.z, a.w), v[2] = pack2(b.x, b.y), v[3] = pack2(b.z, b.w);
}
MOE_DEV void slot_vec(const uint16_t* p, f2 (&v)[4]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack2(bf16_lo(u[i]), bf16_hi(u[i]));
}
MOE_DEV void store_pairs(float* p, const f2 (&v)[4]) {
  const float2 a = unpack2(v[0]), b = unpack2(v[1]), c = unpack2(v[2]), d = unpack2(v[3]);
  reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
  reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
}
MOE_DEV void store_pairs(uint16_t* p, const f2 (&v)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(v[i]);
    u[i] = pack_bf16x2(f.x, f.y);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

template <typename XT, int P, int N, bool STREAM>
__global__ void __launch_bounds__(kRingThreads) layer_norm_bwd_ring_kernel(
    const uint16_t* __restrict__ dy, const XT* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ mean, const float* __restrict__ rstd, const XT* d_stream, int T, int D,
    int stages, XT* dx, float* __restrict__ part, float* __restrict__ dweight,
    float* __restrict__ dbias, unsigned int* dev_err) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kLnMaxStages], empty[kLnMaxStages];
  __shared__ float2 red[2][kLnWarps];
  __shared__ int abort_flag;
  constexpr int kRows = kLnThreads / P;
  const int slot = slot_bytes<XT>(kRows, D, STREAM);
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < stages; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kLnWarps);
    }
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  // the weights beside the ring: it leaves the L1 cache too little for them
  float* wsm = reinterpret_cast<float*>(ring + stages * slot);
  for (int c = threadIdx.x; c < D; c += kRingThreads) wsm[c] = w[c];
  __syncthreads();
  const int turns = (T + kRows - 1) / kRows;
  f2 dw[N][4], db[N][4];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = 0ull;
  const int t = threadIdx.x % P, group = threadIdx.x / P;
  int st = 0;
  uint32_t phase = 0;
  if (threadIdx.x == kLnThreads) {
    // ---- the warp that asks for rows (one lane) ----
    int asked = 0;
    bool ok = true;
    for (int k = blockIdx.x; k < turns; k += gridDim.x) {
      if (!(ok = mbar_wait(smem_u32(&empty[st]), phase ^ 1u, &abort_flag, dev_err))) break;
      const int rows = min(kRows, T - k * kRows);
      const size_t base = static_cast<size_t>(k) * kRows * D;
      const uint32_t bar = smem_u32(&full[st]), dst = smem_u32(ring + st * slot);
      mbar_arrive_expect_tx(bar, slot_bytes<XT>(rows, D, STREAM));
      bulk_load(dst, dy + base, rows * D * 2, bar);
      bulk_load(dst + kRows * D * 2, x + base, rows * D * sizeof(XT), bar);
      if constexpr (STREAM)
        bulk_load(dst + kRows * D * (2 + sizeof(XT)), d_stream + base, rows * D * sizeof(XT), bar);
      ++asked;
      if (++st == stages) st = 0, phase ^= 1u;
    }
    if (!ok) {  // copies may still be on their way into shared memory: another wait for each
      for (int i = 0; i < stages && i < asked; ++i) {
        if (--st < 0) st = stages - 1, phase ^= 1u;
        volatile int local_abort = 0;
        mbar_wait(smem_u32(&full[st]), phase, &local_abort, dev_err);
      }
    }
  }
  const float inv_d = 1.f / static_cast<float>(D);
  int flip = 0;
  float mu1 = 0.f, r1 = 0.f;
  if (threadIdx.x < kLnThreads && blockIdx.x * kRows + group < T)
    mu1 = mean[blockIdx.x * kRows + group], r1 = rstd[blockIdx.x * kRows + group];
  // the rows' warps; each makes every turn of the block, also when a wait was
  // given up (the error word says so), since a row's warps meet at barriers
  for (int k = blockIdx.x; k < turns && threadIdx.x < kLnThreads; k += gridDim.x) {
    const int row = k * kRows + group;
    const bool live = row < T;
    const float mu = mu1, r = r1;
    // the next turn's statistics, a turn ahead
    const int next = min(row + static_cast<int>(gridDim.x) * kRows, T - 1);
    mu1 = mean[next], r1 = rstd[next];
    mbar_wait(smem_u32(&full[st]), phase, &abort_flag, dev_err);
    const uint16_t* sdy = reinterpret_cast<const uint16_t*>(ring + st * slot) + group * D;
    const XT* sx = reinterpret_cast<const XT*>(ring + st * slot + kRows * D * 2) + group * D;
    const XT* sg = sx + kRows * D;
    // n = (x - mu) r and not x r - mu r: that would bring in the rounding of
    // mu r, whatever the size of n (rows 2000 spreads from zero lost 11 bits)
    const f2 rr = pack2(r, r), m0 = pack2(-mu, -mu);
    f2 q1 = 0ull, q2 = 0ull;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * P + t) * 8;
      if (live && c < D) {
        f2 n[4], p[4], wv[4];
        slot_vec(sx + c, n);
        slot_vec(sdy + c, p);
        slot_vec(wsm + c, wv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          n[j] = mul2(add2(n[j], m0), rr);
          dw[i][j] = fma2(p[j], n[j], dw[i][j]);
          db[i][j] = add2(db[i][j], p[j]);
          p[j] = mul2(p[j], wv[j]);
          q1 = add2(q1, p[j]);
          q2 = fma2(p[j], n[j], q2);
        }
      }
    }
    float s1 = unpack2(q1).x + unpack2(q1).y, s2 = unpack2(q2).x + unpack2(q2).y;
    row_sum2<P>(s1, s2, group, red[flip]);
    flip ^= 1;
    // dx = r dy w - r s1 / D - n r s2 / D, the last two as (x - mu) k1 + k0
    const float t2 = -r * s2 * inv_d, t0 = -r * s1 * inv_d;
    const f2 k1 = pack2(t2 * r, t2 * r), k0 = pack2(t0, t0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * P + t) * 8;
      if (live && c < D) {
        f2 n[4], p[4], wv[4];
        slot_vec(sx + c, n);
        slot_vec(sdy + c, p);
        slot_vec(wsm + c, wv);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = fma2(p[j], mul2(wv[j], rr), fma2(add2(n[j], m0), k1, k0));
        if constexpr (STREAM) {
          slot_vec(sg + c, n);
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = add2(p[j], n[j]);
        }
        store_pairs(dx + static_cast<size_t>(row) * D + c, p);
      }
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&empty[st]));
    if (++st == stages) st = 0, phase ^= 1u;
  }
  // every group's sums side by side, then added column by column
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);  // [kRows][2][D]
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * P + t) * 8;
    if (c < D && threadIdx.x < kLnThreads) {
      store_pairs(sums + (group * 2) * D + c, dw[i]);
      store_pairs(sums + (group * 2 + 1) * D + c, db[i]);
    }
  }
  block_sums<kRows>(sums, D, part, dweight, dbias);
}

// out[c] = sum over the nblk partial rows, column c of [2 D]: 32 columns a
// block, kStrips strips of rows, each added in order and then together in order.
constexpr int kStrips = 32;
__global__ void __launch_bounds__(32 * kStrips) layer_norm_reduce_kernel(const float* __restrict__ part, int nblk,
                                                                         int D, float* __restrict__ dweight,
                                                                         float* __restrict__ dbias) {
  __shared__ float strip[kStrips][33];
  griddep_wait();  // the partial rows come from the previous kernel
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v[(kLnMaxPartials + kStrips - 1) / kStrips];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < (kLnMaxPartials + kStrips - 1) / kStrips; ++i) {
    const int b = k + i * kStrips;
    v[i] = c < 2 * D && b < nblk ? part[static_cast<size_t>(b) * 2 * D + c] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < (kLnMaxPartials + kStrips - 1) / kStrips; ++i) s += v[i];
  strip[k][lane] = s;
  __syncthreads();
  // warp k takes column k of the block: 32 strips in a tree of fixed shape
  s = strip[lane][k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int col = blockIdx.x * 32 + k;
  if (lane == 0 && col < 2 * D) {
    if (col < D)
      dweight[col] = s;
    else if (dbias != nullptr)
      dbias[col - D] = s;
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

cudaError_t reduce_partials(const LayerNormBwdArgs& a, int nblk, cudaStream_t s) {
  return launch_kernel(layer_norm_reduce_kernel, dim3((2 * a.D + 31) / 32), dim3(32 * kStrips), 0, s, true,
                       static_cast<const float*>(a.part), nblk, a.D, a.dweight, a.dbias);
}

// A kernel's limit of dynamic shared memory: one for all its calls, whatever
// they ask for, so that host threads with different widths do not take it from
// one another between setting it and launching.  Set once on each device.
constexpr int kMaxDevices = 64;
cudaError_t allow_smem(const void* kernel, size_t limit, bool (&done)[kMaxDevices]) {
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(limit));
  done[dev] = e == cudaSuccess;
  return e;
}

template <typename XT, int P, int N, int VEC>
cudaError_t run_bwd(const LayerNormBwdArgs& a, cudaStream_t s) {
  constexpr int kRows = kLnThreads / P;
  const int sms = current_device_sms();
  int nblk = std::min({(a.T + kRows - 1) / kRows, 2 * sms, kLnMaxPartials});
  cudaError_t e = cudaSuccess;
  if (nblk == 0) return reduce_partials(a, 0, s);  // no rows: the sums are zeros
  static bool smem_set[2][kMaxDevices];            // without and with d_stream
  bool(&set)[kMaxDevices] = smem_set[a.d_stream != nullptr];
  if constexpr (VEC == 1) {
    auto kernel = a.d_stream ? layer_norm_bwd_kernel<XT, P, N, true> : layer_norm_bwd_kernel<XT, P, N, false>;
    const size_t smem = static_cast<size_t>(kRows) * 2 * a.D * sizeof(float);
    constexpr size_t kLimit = static_cast<size_t>(kRows) * 2 * P * N * sizeof(float);  // D <= P N
    if ((e = allow_smem(reinterpret_cast<const void*>(kernel), kLimit, set)) != cudaSuccess) return e;
    e = launch_kernel(kernel, dim3(nblk), dim3(kLnThreads), smem, s, false, static_cast<const uint16_t*>(a.dy),
                      static_cast<const XT*>(a.x), a.weight, a.mean, a.rstd, static_cast<const XT*>(a.d_stream), a.T,
                      a.D, static_cast<XT*>(a.dx), a.part, a.dweight, a.dbias);
  } else {
    // two blocks an SM with at least two slots each, else one
    const size_t slots = slot_bytes<XT>(kRows, a.D, a.d_stream != nullptr), wbytes = a.D * sizeof(float);
    const bool two = 2 * slots + wbytes <= kLnHalfSm;
    const int stages = static_cast<int>(std::min<size_t>(kLnMaxStages, ((two ? kLnHalfSm : kLnWholeSm) - wbytes) / slots));
    const size_t sums = static_cast<size_t>(kRows) * 2 * a.D * sizeof(float);
    const size_t smem = std::max(stages * slots + wbytes, sums);
    if (!two) nblk = std::min(nblk, sms);
    unsigned int* err = nullptr;
    if ((e = device_error_address(&err)) != cudaSuccess) return e;
    auto kernel =
        a.d_stream ? layer_norm_bwd_ring_kernel<XT, P, N, true> : layer_norm_bwd_ring_kernel<XT, P, N, false>;
    if ((e = allow_smem(reinterpret_cast<const void*>(kernel), kLnWholeSm, set)) != cudaSuccess) return e;
    e = launch_kernel(kernel, dim3(nblk), dim3(kRingThreads), smem, s, false, static_cast<const uint16_t*>(a.dy),
                      static_cast<const XT*>(a.x), a.weight, a.mean, a.rstd, static_cast<const XT*>(a.d_stream), a.T,
                      a.D, stages, static_cast<XT*>(a.dx), a.part, a.dweight, a.dbias, err);
  }
  if (e != cudaSuccess || nblk == 1) return e;
  return reduce_partials(a, nblk, s);
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
