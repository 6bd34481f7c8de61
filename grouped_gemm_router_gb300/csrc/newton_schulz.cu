// Newton-Schulz orthogonalisation of stacks of matrices, and the Muon step
// built on it.
//
//   X_0 = G / (|G|_F + eps)                              (G m x n, m <= n)
//   A = X X^T,  B = b A + c A A,  X <- a X + B X         each step
//
// after a few steps the singular values of X are near 1 while its singular
// vectors stay those of G.  A matrix with more rows than columns is worked on
// as its transpose, which the first and the last kernel read and write in
// place of a separate transposition.
//
// Precision.  The products run on the tensor cores with fp16 operands and
// fp32 sums.  fp16 and not bf16 because every operand has a known range
// (singular values below about 1.3, so entries do too): scaled by a power of
// two it holds 3 bits more at the same rate.  The term a X is not part of a
// product and keeps X to 22 bits, as an fp16 value and the fp16 of what it
// leaves (hi + lo).  It matters where G has less than full rank (an expert
// with fewer tokens than rows): what rounding leaves outside the row space
// grows by a in every step, 485-fold in five with a = 3.4445, and nothing
// contracts it.  The products do not need more bits: there A is small.
// Simulated on gradients of rank m/4: 1.1e-2 to 2.6e-2 off without lo,
// 1.9e-3 with it, of which 1.7e-3 is the bf16 rounding of the result (bf16
// operands: 0.9e-1 to 2e-1 without, 0.8e-2 with it).
//
// A and B are symmetric: only the tiles on and below the diagonal are
// computed, and each is stored twice, once transposed.
//
// Every product is a persistent kernel over 256 x 256 tiles, run by CTA pairs
// (tcgen05.mma.cta_group::2, fp32 accumulators in TMEM, operands by TMA with
// the 128-byte swizzle).  Warp roles, the stage ring and the two accumulators
// are those of grouped_gemm.cu.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "moe_device.cuh"
#include "moe_kernels.cuh"

namespace moe {

namespace {

constexpr int kTile = 256;                     // output tile of a CTA pair
constexpr int kBK = 128;                       // k per stage: two 64-wide swizzle atoms
constexpr int kAtomBytes = 128 * 64 * 2;       // 128 rows x 64 k
constexpr int kOperandBytes = 2 * kAtomBytes;  // one operand's half of a stage
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kStages = 3;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kBox = 32;                       // output boxes: 32 rows x 32 columns
constexpr int kBoxBytes = kBox * kBox * 2;
constexpr int kWarpStage = 2 * kBoxBytes;      // staging bytes of an epilogue warp
constexpr int kSmemBytes = kStages * kStageBytes + kEpiWarps * kWarpStage + 1024;
constexpr uint32_t kTmemCols = 512;

// Powers of two that the fp16 copies carry.  X: entries of 1 / sqrt(m n) at
// the start (1.2e-4 for 8192 x 8192) up to about 1.3 stay normal numbers;
// overflow only beyond 16.  A and B: entries of X X^T from 1 / m down, beyond
// 32 overflow.
constexpr float kScaleX = 4096.f;
constexpr float kScaleA = 2048.f;
constexpr float kScaleLo = 2048.f;  // lo = (x - hi) * 2^11, the size of hi again

constexpr int kNormChunks = 256;    // most partial sums of squares of a matrix
constexpr int kNormThreads = 256;

// What a launch computes: A = X X^T, B = b A + c A A, X <- a X + B X, or the
// last of these with the results written.
enum Stage { kGram, kPoly, kApply, kLast };

// ---------------------------------------------------------------------------
// The first two kernels: momentum and norm, then X_0
// ---------------------------------------------------------------------------
struct Source {
  const void* grad;
  float* momentum;
};

MOE_DEV float load_grad(const void* p, bool fp32, size_t i) {
  return fp32 ? static_cast<const float*>(p)[i] : bf16_lo(static_cast<const uint16_t*>(p)[i]);
}

// The stack that matrix `mat` belongs to.
MOE_DEV int stack_of(const NsStacks& st, int mat) {
  int s = 0;
  while (s + 1 < st.n && mat >= st.s[s + 1].first) ++s;
  return s;
}

// m <- mu m + g (with momentum), partial sums of squares of
// u = g, m or g + mu m.  Block (c, mat) takes elements [c, c + 1) * chunk.
__global__ void __launch_bounds__(kNormThreads) ns_norm_kernel(const NsStacks st, const int grad_fp32,
                                                               const float mu, const int nesterov,
                                                               const size_t elems, const size_t chunk,
                                                               float* __restrict__ partial) {
  __shared__ float red[kNormThreads / 32];
  const int mat = blockIdx.y;
  const NsStack& s = st.s[stack_of(st, mat)];
  const size_t base = static_cast<size_t>(mat - s.first) * elems;
  const size_t lo = blockIdx.x * chunk, hi = lo + chunk < elems ? lo + chunk : elems;
  float q = 0.f;
  for (size_t i = lo + threadIdx.x; i < hi; i += kNormThreads) {
    float u = load_grad(s.grad, grad_fp32, base + i);
    if (s.momentum != nullptr) {
      const float m = fmaf(mu, s.momentum[base + i], u);
      s.momentum[base + i] = m;
      u = nesterov ? fmaf(mu, m, u) : m;
    }
    q = fmaf(u, u, q);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = q;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int w = 0; w < kNormThreads / 32; ++w) t += red[w];
    partial[static_cast<size_t>(mat) * kNormChunks + blockIdx.x] = t;
  }
  griddep_launch_dependents();
}

// X_0 in 64 x 64 tiles (zeros past the matrix), transposed for a tall one.
__global__ void __launch_bounds__(256) ns_load_kernel(const NsStacks st, const int grad_fp32, const float mu,
                                                      const int nesterov, const int m, const int n, const int mp,
                                                      const int np, const int chunks, const float eps,
                                                      const float* __restrict__ partial, __half* __restrict__ hi,
                                                      __half* __restrict__ lo) {
  __shared__ float tile[64][65];
  __shared__ float red[8];
  griddep_wait();  // the partial sums and the momentum come from the previous kernel
  const int mat = blockIdx.y;
  const NsStack& s = st.s[stack_of(st, mat)];
  float q = threadIdx.x < chunks ? partial[static_cast<size_t>(mat) * kNormChunks + threadIdx.x] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = q;
  __syncthreads();
  q = red[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) q += red[w];
  // a sum of squares that is no number or past fp32 makes the matrix NaN,
  // which the caller sees, and not a silent zero
  const float inv = q < INFINITY ? kScaleX / (sqrtf(q) + eps) : NAN;
  const int ti = blockIdx.x / (np / 64), tj = blockIdx.x - ti * (np / 64);
  const size_t base = static_cast<size_t>(mat - s.first) * m * n;
  const int a = threadIdx.x >> 6, b = threadIdx.x & 63;
  for (int r = a; r < 64; r += 4) {
    // source row and column: (i, j) of X, or (j, i) of a tall matrix
    const int row = (s.tall ? tj : ti) * 64 + r, col = (s.tall ? ti : tj) * 64 + b;
    const int rows = s.tall ? n : m, cols = s.tall ? m : n;
    float u = 0.f;
    if (row < rows && col < cols) {
      const size_t i = base + static_cast<size_t>(row) * cols + col;
      u = load_grad(s.grad, grad_fp32, i);
      if (s.momentum != nullptr) u = nesterov ? fmaf(mu, s.momentum[i], u) : s.momentum[i];
      u *= inv;
    }
    if (s.tall)
      tile[b][r] = u;
    else
      tile[r][b] = u;
  }
  __syncthreads();
  for (int r = a; r < 64; r += 4) {
    const float u = tile[r][b];
    const __half h = __float2half_rn(u);
    const size_t o = (static_cast<size_t>(mat) * mp + ti * 64 + r) * np + tj * 64 + b;
    hi[o] = h;
    lo[o] = __float2half_rn((u - __half2float(h)) * kScaleLo);
  }
  griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// The products
// ---------------------------------------------------------------------------
struct GemmArgs {
  int count;        // matrices
  int mp, np;       // padded sizes (multiples of 64)
  int m, n;         // sizes
  float a, b, c;    // the step's coefficients
  const __half* A;  // [count, mp, mp]
  const __half* hi;  // X, [count, np]
  const __half* lo;  // or nullptr
  int store_lo;
  NsOutput out;
};

struct Ctl {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// One item of work: tile (ti, tj) of matrix mat.
struct Item {
  int mat, ti, tj;
};

template <bool kTriangle>
MOE_DEV Item item_of(const GemmArgs& p, int idx) {
  const int nt = (p.mp + kTile - 1) / kTile;
  Item it;
  if (!kTriangle) {
    const int ntn = (p.np + kTile - 1) / kTile;
    it.mat = idx / (nt * ntn);
    const int r = idx - it.mat * nt * ntn;
    it.ti = r / ntn;
    it.tj = r - it.ti * ntn;
  } else {
    const int tri = nt * (nt + 1) / 2;
    it.mat = idx / tri;
    int r = idx - it.mat * tri;
    it.ti = 0;
    while (r > it.ti) r -= ++it.ti;
    it.tj = r;
  }
  return it;
}

__host__ __device__ __forceinline__ int item_count(bool triangle, int count, int mp, int np) {
  const int nt = (mp + kTile - 1) / kTile;
  return count * (!triangle ? nt * ((np + kTile - 1) / kTile) : nt * (nt + 1) / 2);
}

MOE_DEV void tma_load_4d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2,
                              int32_t c3, uint64_t cache_policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "l"(cache_policy)
      : "memory");
}

MOE_DEV uint32_t pack_half2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Instruction descriptor of tcgen05.mma.kind::f16: fp16 A (K-major) and B
// (K-major or N-major), fp32 D.
MOE_DEV uint32_t idesc_f16_f32(uint32_t M, uint32_t N, uint32_t b_mn_major) {
  return (1u << 4) | (b_mn_major << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// 32 x 32 fp16 box (lane = row) into the staging buffer, 64-byte swizzle:
// 16-byte chunk c of row r at chunk c ^ ((r / 2) % 4).
MOE_DEV void stage_rows(uint8_t* buf, const float (&v)[32]) {
  const uint32_t lane = lane_id();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(buf + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(pack_half2(v[8 * c], v[8 * c + 1]), pack_half2(v[8 * c + 2], v[8 * c + 3]),
                   pack_half2(v[8 * c + 4], v[8 * c + 5]), pack_half2(v[8 * c + 6], v[8 * c + 7]));
}

// The same box transposed: column j of the box becomes row j.
MOE_DEV void stage_cols(uint8_t* buf, const float (&v)[32]) {
  const uint32_t lane = lane_id();
#pragma unroll
  for (int j = 0; j < 32; ++j)
    *reinterpret_cast<__half*>(buf + j * 64 + (((lane >> 3) ^ ((j >> 1) & 3)) << 4) + (lane & 7) * 2) =
        __float2half_rn(v[j]);
}

// 32 consecutive halves as floats, through L2.
MOE_DEV void load_halves(const __half* p, float (&v)[32]) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 u = __ldcg(q + c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      v[8 * c + 2 * k] = f.x;
      v[8 * c + 2 * k + 1] = f.y;
    }
  }
}

// Element (row, col) of the stack's own matrix: the orthogonalised value o
// is the result, or moves the weight.
MOE_DEV void write_result(const NsOutput& o, const NsStack& s, size_t at, float v) {
  if (o.kind == kNsPlain) {
    static_cast<uint16_t*>(s.weight)[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
  } else if (o.kind == kNsWeightBf16) {
    uint16_t* w = static_cast<uint16_t*>(s.weight) + at;
    *w = static_cast<uint16_t>(pack_bf16x2(fmaf(bf16_lo(*w), o.keep, -o.step * v), 0.f));
  } else {
    float* w = static_cast<float*>(s.weight) + at;
    const float t = fmaf(*w, o.keep, -o.step * v);
    *w = t;
    if (s.weight_bf16 != nullptr) static_cast<uint16_t*>(s.weight_bf16)[at] = static_cast<uint16_t>(pack_bf16x2(t, 0.f));
  }
}

// mapP: the left operand, mapQ: the right one, mapOut: the product's fp16
// output (A, B or X's hi), mapLo: X's lo.
template <Stage kStage>
__global__ void __launch_bounds__(kThreads, 1)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap mapP, const __grid_constant__ CUtensorMap mapQ,
                   const __grid_constant__ CUtensorMap mapOut, const __grid_constant__ CUtensorMap mapLo,
                   const __grid_constant__ GemmArgs p, const __grid_constant__ NsStacks st,
                   unsigned int* const dev_err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t smem_base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(cluster_id_x()), npairs = static_cast<int>(num_clusters_x());
  constexpr bool kTriangle = kStage == kGram || kStage == kPoly;
  const int K = kStage == kGram ? p.np : p.mp;
  const int nkb = (K + kBK - 1) / kBK;
  const int total = item_count(kTriangle, p.count, p.mp, p.np);

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&mapP);
    tma_prefetch_desc(&mapQ);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&ctl.full[i]), 1);
      mbar_init(smem_u32(&ctl.empty[i]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ctl.tfull[b]), 1);
      mbar_init(smem_u32(&ctl.tempty[b]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(&ctl.drain), 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&ctl.tmem_base), kTmemCols);
    tmem_relinquish_pair();
    tc_fence_before_sync();
  }
  griddep_launch_dependents();
  griddep_wait();  // the operands come from earlier kernels
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem_base = ctl.tmem_base;
  volatile int* abort_flag = &ctl.abort;

  if (warp == 0) {
    // ===================== TMA producer (both CTAs) =====================
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_normal();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int idx = pair; idx < total && ok; idx += npairs) {
        const Item it = item_of<kTriangle>(p, idx);
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_cluster(smem_u32(&ctl.empty[stage]), phase ^ 1u, abort_flag, dev_err)) {
            ok = false;
            break;
          }
          const uint32_t bar = map_to_cta(smem_u32(&ctl.full[stage]), 0);
          const uint32_t sp = smem_base + stage * kStageBytes, sq = sp + kOperandBytes;
          // both CTAs' boxes count in full, rows and k past the matrix are zeros
          if (leader) mbar_arrive_expect_tx(smem_u32(&ctl.full[stage]), 2 * kStageBytes);
          tma_load_4d_pair(sp, &mapP, bar, 0, it.ti * kTile + 128 * rank, kb * (kBK / 64), it.mat, policy);
          if (!kTriangle)
            tma_load_4d_pair(sq, &mapQ, bar, 0, kb * kBK, it.tj * (kTile / 64) + 2 * rank, it.mat, policy);
          else
            tma_load_4d_pair(sq, &mapQ, bar, 0, it.tj * kTile + 128 * rank, kb * (kBK / 64), it.mat, policy);
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) {
        // Let the copies already in flight land before the CTA exits.
        for (int i = 0; i < kStages && i < issued; ++i) {
          if (--stage < 0) {
            stage = kStages - 1;
            phase ^= 1u;
          }
          volatile int local_abort = 0;
          mbar_wait_cluster(smem_u32(&ctl.full[stage]), phase, &local_abort, dev_err);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ===================== MMA issuer (leader only) =====================
    if (lane == 0 && leader) {
      constexpr bool n_major = !kTriangle;
      const uint32_t idesc = idesc_f16_f32(kTile, kTile, n_major ? 1u : 0u);
      int stage = 0, i = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int idx = pair; idx < total && ok; idx += npairs, ++i) {
        const int buf = i & 1;
        if (!mbar_wait_cluster(smem_u32(&ctl.tempty[buf]), ((i >> 1) & 1) ^ 1u, abort_flag, dev_err)) break;
        tc_fence_after_sync();
        const uint32_t d = tmem_base + buf * kTile;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_cluster(smem_u32(&ctl.full[stage]), phase, abort_flag, dev_err)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sp = smem_base + stage * kStageBytes, sq = sp + kOperandBytes;
          const int slices = K - kb * kBK >= kBK ? kBK / 16 : 4;  // K is a multiple of 64
          for (int kk = 0; kk < slices; ++kk) {
            const uint32_t off = (kk >> 2) * kAtomBytes + (kk & 3) * 32;
            const uint64_t pd = smem_desc_sw128(sp + off, 16, 1024);
            const uint64_t qd = n_major ? smem_desc_sw128(sq + kk * 2048, kAtomBytes, 1024)
                                        : smem_desc_sw128(sq + off, 16, 1024);
            umma_bf16_pair(d, pd, qd, idesc, (kb | kk) != 0 ? 1u : 0u);
          }
          umma_commit_pair(smem_u32(&ctl.empty[stage]), 0x3);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(smem_u32(&ctl.tfull[buf]), 0x3);
      }
      umma_commit_pair(smem_u32(&ctl.drain), 0x1);
      volatile int local_abort = 0;
      mbar_wait_cluster(smem_u32(&ctl.drain), 0, &local_abort, dev_err);
    }
    __syncwarp();
  } else {
    // ===================== epilogue (both CTAs) =====================
    // Warp w: TMEM lanes 32 (w % 4) .. + 31 and half (w - 2) / 4 of the columns.
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t tempty0 = map_to_cta(smem_u32(&ctl.tempty[0]), 0);
    const uint32_t tempty1 = map_to_cta(smem_u32(&ctl.tempty[1]), 0);
    uint8_t* buf0 = smem + kStages * kStageBytes + (warp - 2) * kWarpStage;
    uint8_t* buf1 = buf0 + kBoxBytes;
    const int ncols = kTriangle ? p.mp : p.np;
    // boxes read from TMEM at a time: all four where the epilogue holds
    // little else (the accumulator is free again the sooner), else two
    constexpr int kBurst = kStage == kGram ? 4 : 2;
    int i = 0;
    for (int idx = pair; idx < total; idx += npairs, ++i) {
      const Item it = item_of<kTriangle>(p, idx);
      const int buf = i & 1;
      const bool got = mbar_wait_cluster(smem_u32(&ctl.tfull[buf]), (i >> 1) & 1, abort_flag, dev_err);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after_sync();
      const int row0 = it.ti * kTile + 128 * static_cast<int>(rank) + q * 32;
      const int col0 = it.tj * kTile + part * 128;
      // padded sizes are multiples of 64: a box is inside or outside
      const int nbox = row0 < p.mp && col0 < ncols ? min(4, (ncols - col0) / kBox) : 0;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kTile + part * 128;
      uint32_t acc[kBurst][32];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (b % kBurst == 0) {
#pragma unroll
          for (int j = 0; j < kBurst; ++j)
            if (b + j < nbox) tmem_ld_32cols(taddr + (b + j) * kBox, acc[j]);
          if (b < nbox) tmem_ld_wait();
          if (b + kBurst >= 4) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(buf ? tempty1 : tempty0);
          }
        }
        if (b >= nbox) continue;
        const int col = col0 + b * kBox;
        float v[32];
        if constexpr (kStage == kGram) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(acc[b % kBurst][j]) * (kScaleA / (kScaleX * kScaleX));
        } else if constexpr (kStage == kPoly) {
          load_halves(p.A + (static_cast<size_t>(it.mat) * p.mp + row0 + lane) * p.mp + col, v);
          const float c = p.c / kScaleA;
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = fmaf(c, __uint_as_float(acc[b % kBurst][j]), p.b * v[j]);
        } else {
          const size_t at = (static_cast<size_t>(it.mat) * p.mp + row0 + lane) * p.np + col;
          load_halves(p.hi + at, v);
          if (p.lo != nullptr) {
            float l[32];
            load_halves(p.lo + at, l);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = fmaf(1.f / kScaleLo, l[j], v[j]);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = fmaf(p.a, v[j], __uint_as_float(acc[b % kBurst][j]) * (1.f / kScaleA));
        }
        bulk_wait_group_read0();  // lane 0's stores have read the buffers
        __syncwarp();
        if constexpr (kStage == kLast) {
          // results, 32 consecutive elements of the stack's own rows at a time
          const NsStack& s = st.s[stack_of(st, it.mat)];
          const size_t base = static_cast<size_t>(it.mat - s.first) * p.m * p.n;
          if (s.tall) {  // column j of the box is a run of row j: lanes are consecutive
            if (row0 + lane < p.m) {
#pragma unroll 4
              for (int j = 0; j < 32; ++j)
                if (col + j < p.n)
                  write_result(p.out, s, base + static_cast<size_t>(col + j) * p.m + row0 + lane, v[j] * (1.f / kScaleX));
            }
          } else {  // turn the box so that lanes are columns
            float* f = reinterpret_cast<float*>(buf0);
#pragma unroll
            for (int j = 0; j < 32; ++j) f[lane * 32 + (j ^ lane)] = v[j];
            __syncwarp();
            if (col + lane < p.n) {
#pragma unroll 4
              for (int r = 0; r < 32; ++r)
                if (row0 + r < p.m)
                  write_result(p.out, s, base + static_cast<size_t>(row0 + r) * p.n + col + lane,
                               f[r * 32 + (lane ^ r)] * (1.f / kScaleX));
            }
            __syncwarp();
          }
        } else {
          stage_rows(buf0, v);
          const bool mirror = kTriangle && it.ti != it.tj;
          if (mirror) stage_cols(buf1, v);
          const bool low = kStage == kApply && p.store_lo;
          if (low) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = (v[j] - __half2float(__float2half_rn(v[j]))) * kScaleLo;
            stage_rows(buf1, v);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&mapOut, smem_u32(buf0), col, row0, it.mat);
            if (mirror) tma_store_3d(&mapOut, smem_u32(buf1), row0, col, it.mat);
            if (low) tma_store_3d(&mapLo, smem_u32(buf1), col, row0, it.mat);
            bulk_commit_group();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group0();
    __syncwarp();
  }
  tc_fence_before_sync();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
inline size_t align_up(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int pad64(int v) { return (v + 63) / 64 * 64; }

struct Buffers {
  float* partial;
  __half *hi[2], *lo[2], *A, *B;
  size_t bytes;
};

Buffers carve(void* base, int count, int mp, int np) {
  Buffers w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align_up(bytes);
    return base ? static_cast<char*>(base) + o : nullptr;
  };
  const size_t x = static_cast<size_t>(count) * mp * np * 2, a = static_cast<size_t>(count) * mp * mp * 2;
  w.partial = reinterpret_cast<float*>(take(static_cast<size_t>(count) * kNormChunks * 4));
  for (int i = 0; i < 2; ++i) w.hi[i] = reinterpret_cast<__half*>(take(x));
  for (int i = 0; i < 2; ++i) w.lo[i] = reinterpret_cast<__half*>(take(x));
  w.A = reinterpret_cast<__half*>(take(a));
  w.B = reinterpret_cast<__half*>(take(a));
  w.bytes = off;
  return w;
}

struct Setup {
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  int pairs[64] = {0};
};
Setup g_setup;
std::mutex g_setup_mu;

// The encoder and the co-resident pairs of the current device.
cudaError_t setup(PFN_cuTensorMapEncodeTiled_v12000* encode, int* pairs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_setup_mu);
  if (g_setup.encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
    g_setup.encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  if (g_setup.pairs[dev] == 0) {
    const void* fns[] = {
        reinterpret_cast<const void*>(ns_gemm_kernel<kGram>), reinterpret_cast<const void*>(ns_gemm_kernel<kPoly>),
        reinterpret_cast<const void*>(ns_gemm_kernel<kApply>), reinterpret_cast<const void*>(ns_gemm_kernel<kLast>)};
    for (const void* fn : fns) {
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      if (e != cudaSuccess) return e;
    }
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (sms / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, fns[kGram], &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    g_setup.pairs[dev] = n;
  }
  *encode = g_setup.encode;
  *pairs = g_setup.pairs[dev];
  return cudaSuccess;
}

// [count, rows, cols] fp16 (cols a multiple of 64) viewed as {64 columns,
// rows, cols / 64, count}: a box is 128 rows of two 64-column blocks, each
// block 16 KB with the 128-byte swizzle.  It serves a K-major operand (128
// rows, 128 k) and an N-major one (128 k, 128 columns) alike.
cudaError_t operand_map(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* p, int count, int rows,
                        int cols) {
  cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / 64),
                        static_cast<cuuint64_t>(count)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(cols) * 2, 128, static_cast<cuuint64_t>(rows) * cols * 2};
  cuuint32_t box[4] = {64, 128, 2, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(p), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// [count, rows, cols] fp16 for stores of 32 x 32 boxes.
cudaError_t store_map(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* p, int count, int rows,
                      int cols) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(count)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(rows) * cols * 2};
  cuuint32_t box[3] = {kBox, kBox, 1};
  cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <Stage kStage>
cudaError_t launch_gemm(int pairs, const CUtensorMap& P, const CUtensorMap& Q, const CUtensorMap& out,
                        const CUtensorMap& lo, const GemmArgs& a, const NsStacks& st, unsigned int* err,
                        cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * std::min(pairs, item_count(kStage == kGram || kStage == kPoly, a.count, a.mp, a.np)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, ns_gemm_kernel<kStage>, P, Q, out, lo, a, st, err);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t ns_workspace_bytes(int count, int m, int n) { return carve(nullptr, count, pad64(m), pad64(n)).bytes; }

cudaError_t launch_newton_schulz(const NsProblem& pr, void* workspace, cudaStream_t s) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  int pairs = 0;
  unsigned int* err = nullptr;
  cudaError_t e = setup(&enc, &pairs);
  if (e != cudaSuccess) return e;
  if ((e = device_error_address(&err)) != cudaSuccess) return e;
  const int mp = pad64(pr.m), np = pad64(pr.n), count = pr.count;
  const Buffers w = carve(workspace, count, mp, np);

  const size_t elems = static_cast<size_t>(pr.m) * pr.n;
  size_t chunk = (elems + kNormChunks - 1) / kNormChunks;
  if (chunk < 8192) chunk = 8192;
  const int chunks = static_cast<int>((elems + chunk - 1) / chunk);
  e = launch_kernel(ns_norm_kernel, dim3(chunks, count), dim3(kNormThreads), 0, s, false, pr.stacks, pr.grad_fp32,
                    pr.momentum, pr.nesterov, elems, chunk, w.partial);
  if (e != cudaSuccess) return e;
  e = launch_kernel(ns_load_kernel, dim3((mp / 64) * (np / 64), count), dim3(256), 0, s, true, pr.stacks,
                    pr.grad_fp32, pr.momentum, pr.nesterov, pr.m, pr.n, mp, np, chunks, pr.eps,
                    static_cast<const float*>(w.partial), w.hi[0], w.lo[0]);
  if (e != cudaSuccess) return e;

  CUtensorMap mX[2], sX[2], sLo[2], mA, sA, mB, sB;
  for (int i = 0; i < 2; ++i) {
    if ((e = operand_map(enc, &mX[i], w.hi[i], count, mp, np)) != cudaSuccess) return e;
    if ((e = store_map(enc, &sX[i], w.hi[i], count, mp, np)) != cudaSuccess) return e;
    if ((e = store_map(enc, &sLo[i], w.lo[i], count, mp, np)) != cudaSuccess) return e;
  }
  if ((e = operand_map(enc, &mA, w.A, count, mp, mp)) != cudaSuccess) return e;
  if ((e = store_map(enc, &sA, w.A, count, mp, mp)) != cudaSuccess) return e;
  if ((e = operand_map(enc, &mB, w.B, count, mp, mp)) != cudaSuccess) return e;
  if ((e = store_map(enc, &sB, w.B, count, mp, mp)) != cudaSuccess) return e;

  for (int k = 0; k < pr.steps; ++k) {
    const int cur = k & 1;
    GemmArgs a{};
    a.count = count;
    a.mp = mp, a.np = np, a.m = pr.m, a.n = pr.n;
    a.a = pr.coeff[k][0], a.b = pr.coeff[k][1], a.c = pr.coeff[k][2];
    a.A = w.A;
    a.hi = w.hi[cur];
    a.lo = w.lo[cur];
    a.store_lo = 1;
    a.out = pr.out;
    if ((e = launch_gemm<kGram>(pairs, mX[cur], mX[cur], sA, sA, a, pr.stacks, err, s)) != cudaSuccess) return e;
    if ((e = launch_gemm<kPoly>(pairs, mA, mA, sB, sB, a, pr.stacks, err, s)) != cudaSuccess) return e;
    if (k + 1 < pr.steps)
      e = launch_gemm<kApply>(pairs, mB, mX[cur], sX[cur ^ 1], sLo[cur ^ 1], a, pr.stacks, err, s);
    else
      e = launch_gemm<kLast>(pairs, mB, mX[cur], sX[cur], sX[cur], a, pr.stacks, err, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
