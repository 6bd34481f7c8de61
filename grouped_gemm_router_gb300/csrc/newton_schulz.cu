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
// two it holds 3 bits more at the same rate.  Two things are kept apart:
//  * The term a X is not part of a product and keeps X to about 14 bits, as
//    fp16 and what that leaves in e5m2 (hi + lo; not for the last step's
//    X).  e5m2 is the upper byte of an fp16, so it needs no scale and is
//    cheap to widen.  It matters where G has less than full rank (an expert
//    with fewer tokens than rows): what rounding leaves outside the row space
//    grows by a in every step, 485-fold in five with a = 3.4445, and nothing
//    contracts it.  The products need no more bits there: A is small.
//  * In the last two steps B is close to -2.7 I and cancels most of a X, so
//    the rounding of its diagonal would be the largest error left.  There the
//    diagonal goes from product to product in fp32 and the stored B has
//    zeros in its place.  (Not before: it would split what cancels outside
//    the row space into two differently rounded halves.)
// Simulated 2-norm errors, of which the bf16 rounding of the result is
// 1.66e-3: full rank 1.8e-3 to 2.1e-3 (2.3e-3 to 2.6e-3 without the fp32
// diagonal), rank m/4 2.0e-3 (1.1e-2 to 2.6e-2 without lo; with bf16 operands
// 0.9e-1 to 2e-1).  Measured before that rounding, five steps: 0.6e-3 (4096 x
// 4096) to 1.3e-3 (65 x 200) at full rank, 1.0e-3 to 1.6e-3 at rank m/4.  The
// roundings of X (in A and in B X), A and B share it about evenly, over all
// steps: simulated, leaving out any one of them takes off a tenth to a fifth.
// So a result as exact as fp32 products would take operands split in two, three
// products for each one here; the update that this is for has far more noise.
//
// A and B are symmetric: only the tiles on and below the diagonal are computed
// and stored.  Where a product needs one from above, it loads the tile from
// below as the transposed (M- or N-major) operand, which costs nothing.
//
// What only the epilogues read (lo, and a copy of A) is kept in the order in
// which they hold it: for each warp and 32 x 32 box, 32-byte pieces of 32
// lanes side by side.  So those accesses are whole lines and need no turning
// in shared memory, whose bandwidth the products use.  The operands, hi among
// them, come and go by TMA.
//
// All products of all steps are one persistent launch over 256 x 256 tiles
// (256 x 128 where there are few),
// run by CTA pairs (tcgen05.mma.cta_group::2, fp32 accumulators in TMEM,
// operands by TMA with the 128-byte swizzle).  The tiles of all (product,
// matrix) are numbered product by product and pair p takes tiles p, p +
// pairs, ...  A tile waits until the product that it reads, of its own
// matrix only, is complete (a counter per product and matrix), so one
// product's last tiles run beside the next one's first.  The order makes
// every tile depend on lower-numbered ones only and the launch is
// cooperative, so the waits end; they are bounded all the same.
//
// Measured, whole calls: 24 matrices of 768 x 1536 513 us (0.74 PFLOP/s of the
// operations that symmetry leaves), 12 of 2048 x 8192 5.6 ms (1.19, at the
// power limit), 8 of 768 x 1536 without the step's weights 218 us.  Of the 513
// us the kernels before the products take about 98, near the memory's rate.
// With the epilogues taken out an earlier state's 509 became 354: what bounds
// these sizes is the epilogues' traffic and the way from product to product.
//
// Warp roles (one CTA per SM):
//   warp 0      TMA producer (one lane) -- both CTAs load their own halves
//   warp 1      TMEM allocator; MMA issuer (one lane, leader only)
//   warps 2-17  epilogue
//   warp 18     counts the tiles whose results are in memory
//   warp 19     finds the CTA's next tiles, waits for what they depend on and
//               posts them for the others, a few ahead
#include <cuda_fp16.h>
#include <cuda_fp8.h>
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
constexpr int kEpiWarps = 16;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kBox = 32;                       // columns an epilogue warp takes from TMEM at a time
constexpr int kWarpStage = kBox * kBox * 2;    // its box in shared memory, fp16 (or 16 rows in fp32)
constexpr int kBoxX = 2 * 512;                 // its box of lo: 8 words a lane
constexpr int kBoxA = 4 * 512;                 // its box of A: 16 words a lane
constexpr int kSmemBytes = kStages * kStageBytes + kEpiWarps * kWarpStage + 1024;
constexpr uint32_t kTmemCols = 512;

// The power of two that the fp16 copies of X carry: entries of 1 / sqrt(m n)
// at the start (1.2e-4 for 8192 x 8192) up to about 1.3 stay normal numbers;
// overflow only beyond 16.  A and B carry none: their entries count beside
// the a of a X, so fp16's smallest step, 6e-8, is enough.
constexpr float kScaleX = 4096.f;

constexpr int kNormChunks = 256;    // most partial sums of squares of a matrix
constexpr int kNormThreads = 256;

// The products of a step: A = X X^T, B = b A + c A A, X <- a X + B X.
enum Product { kGram, kPoly, kApply };

// ---------------------------------------------------------------------------
// The first two kernels: momentum and norm, then X_0
// ---------------------------------------------------------------------------
// The stack that matrix `mat` belongs to.
MOE_DEV int stack_of(const NsStacks& st, int mat) {
  int s = 0;
  while (s + 1 < st.n && mat >= st.s[s + 1].first) ++s;
  return s;
}

// VEC consecutive values (4: one 16- or 8-byte load).
template <int VEC>
MOE_DEV void load_vals(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  } else {
    v[0] = *p;
  }
}
template <int VEC>
MOE_DEV void load_vals(const uint16_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
  } else {
    v[0] = bf16_lo(*p);
  }
}

// m <- mu m + g (with momentum), partial sums of squares of u = g, m or
// g + mu m.  Block (c, mat) takes elements [c, c + 1) * chunk; the first of a
// matrix also clears its counters.
template <typename GT, int VEC>
__global__ void __launch_bounds__(kNormThreads) ns_norm_kernel(const __grid_constant__ NsStacks st, const float mu,
                                                               const int nesterov, const size_t elems,
                                                               const size_t chunk, float* __restrict__ partial,
                                                               unsigned int* __restrict__ done, const int products) {
  __shared__ float red[kNormThreads / 32];
  const int mat = blockIdx.y;
  const NsStack& s = st.s[stack_of(st, mat)];
  const size_t base = static_cast<size_t>(mat - s.first) * elems;
  const GT* g = static_cast<const GT*>(s.grad) + base;
  float* mom = s.momentum ? s.momentum + base : nullptr;
  const size_t lo = blockIdx.x * chunk, hi = lo + chunk < elems ? lo + chunk : elems;
  if (blockIdx.x == 0 && threadIdx.x < products) done[static_cast<size_t>(mat) * products + threadIdx.x] = 0;
  float q = 0.f;
  constexpr int kStep = kNormThreads * VEC, kUnroll = 4;
  for (size_t i0 = lo + threadIdx.x * VEC; i0 < hi; i0 += kStep * kUnroll) {
    float u[kUnroll][VEC], m[kUnroll][VEC];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const size_t i = i0 + k * kStep;
      if (i < hi) {
        load_vals<VEC>(g + i, u[k]);
        if (mom != nullptr) load_vals<VEC>(mom + i, m[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const size_t i = i0 + k * kStep;
      if (i >= hi) continue;
      if (mom != nullptr) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          m[k][j] = fmaf(mu, m[k][j], u[k][j]);
          u[k][j] = nesterov ? fmaf(mu, m[k][j], u[k][j]) : m[k][j];
        }
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(mom + i) = make_float4(m[k][0], m[k][1], m[k][2], m[k][3]);
        else
          mom[i] = m[k][0];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) q = fmaf(u[k][j], u[k][j], q);
    }
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

MOE_DEV uint32_t pack_half2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

MOE_DEV float2 unpack_half2(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }

MOE_DEV float half_minus(uint32_t h, float c) {  // the low half of h, minus c, in fp32
  float d;
  asm("sub.f32.f16 %0, %1, %2;" : "=f"(d) : "h"(static_cast<uint16_t>(h)), "f"(c));
  return d;
}

// lo is kept with its sign turned, as hi - x: that is one instruction, and so
// is x = hi - lo.
MOE_DEV uint32_t pack_lo2(float a, float b, uint32_t h) {
  return __nv_cvt_float2_to_fp8x2(make_float2(half_minus(h, a), half_minus(h >> 16, b)), __NV_SATFINITE, __NV_E5M2);
}

// Four values from two packed pairs of hi and four bytes of lo.
MOE_DEV void unpack_hi_lo4(uint32_t h01, uint32_t h23, uint32_t lo, float (&x)[4]) {
  const float2 l01 = unpack_half2(__byte_perm(lo, 0, 0x1404)), l23 = unpack_half2(__byte_perm(lo, 0, 0x3424));
  x[0] = half_minus(h01, l01.x), x[1] = half_minus(h01 >> 16, l01.y);
  x[2] = half_minus(h23, l23.x), x[3] = half_minus(h23 >> 16, l23.y);
}

// The number of the 32 x 32 box at (i, j) of matrix mat; rows and cols padded.
MOE_DEV size_t box_number(int mat, int rows, int cols, int i, int j) {
  return (static_cast<size_t>(mat) * (rows / kBox) + i / kBox) * (cols / kBox) + j / kBox;
}

// X_0 in 64 x 64 tiles (zeros past the matrix), transposed for a tall one.
template <typename GT, int VEC>
__global__ void __launch_bounds__(256) ns_load_kernel(const __grid_constant__ NsStacks st, const float mu,
                                                      const int nesterov, const int m, const int n, const int mp,
                                                      const int np, const int chunks, const float eps,
                                                      const float* __restrict__ partial, __half* __restrict__ hi,
                                                      uint8_t* __restrict__ lo) {
  __shared__ float tile[64][65];
  __shared__ float red[8];
  griddep_wait();  // the partial sums and the momentum come from the previous kernel
  const int mat = blockIdx.y;
  const NsStack& s = st.s[stack_of(st, mat)];
  const int ti = blockIdx.x / (np / 64), tj = blockIdx.x - ti * (np / 64);
  const size_t base = static_cast<size_t>(mat - s.first) * m * n;
  const GT* g = static_cast<const GT*>(s.grad) + base;
  const float* mom = s.momentum ? s.momentum + base : nullptr;
  // source tile: rows and columns of the stack's own matrix
  const int rows = s.tall ? n : m, cols = s.tall ? m : n;
  const int r0 = (s.tall ? tj : ti) * 64, c0 = (s.tall ? ti : tj) * 64;
  constexpr int kPerRow = 64 / VEC, kRows = 256 / kPerRow, kTurns = 64 / kRows;
  const int tr = threadIdx.x / kPerRow, tc = threadIdx.x % kPerRow * VEC;
  float u[kTurns][VEC];
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int row = r0 + tr + k * kRows, col = c0 + tc;
#pragma unroll
    for (int j = 0; j < VEC; ++j) u[k][j] = 0.f;
    if (row < rows && col < cols) {
      const size_t i = static_cast<size_t>(row) * cols + col;
      if (mom == nullptr) {
        load_vals<VEC>(g + i, u[k]);
      } else {
        load_vals<VEC>(mom + i, u[k]);
        if (nesterov) {
          float v[VEC];
          load_vals<VEC>(g + i, v);
#pragma unroll
          for (int j = 0; j < VEC; ++j) u[k][j] = fmaf(mu, u[k][j], v[j]);
        }
      }
    }
  }
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
#pragma unroll
  for (int k = 0; k < kTurns; ++k)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int r = tr + k * kRows, c = tc + j;
      const float v = r0 + r < rows && c0 + c < cols ? u[k][j] * inv : 0.f;
      if (s.tall)
        tile[c][r] = v;
      else
        tile[r][c] = v;
    }
  __syncthreads();
  const int wr = threadIdx.x >> 4, wc = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int r = wr; r < 64; r += 16) {
    const float a = tile[r][wc], b = tile[r][wc + 1], c = tile[r][wc + 2], d = tile[r][wc + 3];
    const size_t o = (static_cast<size_t>(mat) * mp + ti * 64 + r) * np + tj * 64 + wc;
    *reinterpret_cast<uint2*>(hi + o) = make_uint2(pack_half2(a, b), pack_half2(c, d));
  }
  // lo: four boxes, two warps each, a lane a row of 16 columns
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int br = (w >> 1 & 1) * 32, bc = (w >> 2) * 32, half = w & 1;
  uint32_t word[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float* v = &tile[br + lane][bc + 16 * half + 4 * k];
    word[k] = pack_lo2(v[0], v[1], pack_half2(v[0], v[1])) | (pack_lo2(v[2], v[3], pack_half2(v[2], v[3])) << 16);
  }
  uint8_t* box = lo + box_number(mat, mp, np, ti * 64 + br, tj * 64 + bc) * kBoxX;
  *reinterpret_cast<uint4*>(box + lane * 32 + half * 16) = make_uint4(word[0], word[1], word[2], word[3]);
}

// ---------------------------------------------------------------------------
// The products
// ---------------------------------------------------------------------------
struct GemmArgs {
  int count;        // matrices
  int group;        // of them, that are worked on at a time
  int steps;
  int mp, np;       // padded sizes (multiples of 64)
  int m, n;         // sizes
  int tn;           // columns of a tile: 256, or 128
  int direct;       // each epilogue warp counts its part of a tile itself
  float coeff[MOE_MAX_NS_STEPS][3];
  const __half* hi[2];  // X, [count, mp, np], in turns
  uint8_t* lo;      // what hi leaves of X, in boxes
  uint8_t* a;       // the epilogues' copy of A, in boxes
  float* diag;      // [count, mp]: B's diagonal where it is kept apart
  unsigned int* done;  // [count, 3 * steps] CTAs' (or warps') parts of tiles that are complete
  NsOutput out;
};

struct NsMaps {
  CUtensorMap X[2], A, B;           // operands: 128 rows x two 64-column blocks
  CUtensorMap boxX[2], boxA, boxB;  // the same arrays in 32 x 32 boxes
};

// A tile as it is posted: the product (-1: there are no more), matrix, place.
struct Tile {
  int prod, mat, ti, tj;
};
constexpr int kPosted = 8;  // tiles posted at a time

struct Ctl {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint64_t box[kEpiWarps];
  uint32_t tmem_base;
  int abort;
  int ready;                // tiles posted: what they read is complete
  int written[kEpiWarps];   // tiles whose stores an epilogue warp has issued
  int counted;              // tiles that all warps are done with
  Tile tile[kPosted];
};

// Walks the tiles of one pair in the common order: group of matrices after
// group, in a group product after product, in a product matrix after matrix.
struct Walk {
  int first, g0, prod;     // number of the product's first tile, group, product
  int mat, ti, tj;         // the tile
  MOE_DEV Walk() : first(0), g0(0), prod(0) {}
  // Tiles in row ti of a matrix in product `prod`: a symmetric one's up to the
  // 256 columns that hold the diagonal.
  __host__ MOE_DEV static int row_tiles(const GemmArgs& p, int prod, int ti) {
    const int all = ((prod % 3 == kApply ? p.np : p.mp) + p.tn - 1) / p.tn;
    return prod % 3 == kApply ? all : min(all, (ti + 1) * (kTile / p.tn));
  }
  // Tiles of one matrix in product `prod`.
  __host__ MOE_DEV static int tiles(const GemmArgs& p, int prod) {
    const int nt = (p.mp + kTile - 1) / kTile;
    if (prod % 3 == kApply) return nt * row_tiles(p, prod, 0);
    return nt * (nt - 1) / 2 * (kTile / p.tn) + row_tiles(p, prod, nt - 1);  // all rows but the last are whole
  }
  // Moves to tile `idx`; false past the last one.  idx never decreases.
  MOE_DEV bool to(const GemmArgs& p, int idx) {
    for (; g0 < p.count; g0 += p.group, prod = 0)
      for (; prod < 3 * p.steps; ++prod) {
        const int per = tiles(p, prod), here = min(p.group, p.count - g0) * per;
        if (idx < first + here) {
          int r = idx - first;
          mat = g0 + r / per;
          r %= per;
          for (ti = 0; r >= row_tiles(p, prod, ti); ++ti) r -= row_tiles(p, prod, ti);
          tj = r;
          return true;
        }
        first += here;
      }
    return false;
  }
};

// A wait's turn: false when it is to be given up, because another thread of
// the CTA has or because it has lasted too long.
MOE_DEV bool keep_waiting(uint32_t it, uint64_t& t0, volatile int* abort, unsigned int* dev_err) {
  if ((it & 63u) != 63u) return true;
  if (*abort) return false;
  const uint64_t t = global_timer_ns();
  if (t0 == 0) t0 = t;
  if (t - t0 <= MOE_WAIT_TIMEOUT_NS) return true;
  *abort = 1;
  atomicOr(dev_err, MOE_DEVERR_TIMEOUT);
  return false;
}

// Waits until the product before `prod` of matrix `mat` is complete, and
// makes its results visible to this thread's loads and TMA operations.
MOE_DEV bool wait_product(const GemmArgs& p, int prod, int mat, volatile int* abort, unsigned int* dev_err) {
  if (prod == 0) return true;  // X_0 comes from an earlier kernel
  const unsigned int* c = p.done + static_cast<size_t>(mat) * 3 * p.steps + prod - 1;
  const unsigned int target = Walk::tiles(p, prod - 1) * 2 * (p.direct ? kEpiWarps : 1);
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(c) : "memory");
    if (v >= target) break;
    if (!keep_waiting(it, t0, abort, dev_err)) return false;
  }
  asm volatile("fence.proxy.async.global;" ::: "memory");
  return true;
}

// Counts a part of tile t as complete, after all that this thread has seen
// written.
MOE_DEV void count_done(const GemmArgs& p, const Tile& t) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.done + static_cast<size_t>(t.mat) * 3 * p.steps + t.prod)
               : "memory");
}

// Counters in shared memory, written by one thread each.
MOE_DEV void count_store(int* c, int v) {
  asm volatile("st.release.cta.shared.s32 [%0], %1;" ::"r"(smem_u32(c)), "r"(v) : "memory");
}

// Waits until *c is above i; returns it, or -1 when the wait was given up.
// What the writer has acquired or stored before, this thread may read.
MOE_DEV int wait_count(const int* c, int i, volatile int* abort, unsigned int* dev_err) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    int v;
    asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(c)) : "memory");
    if (v > i) return v;
    if (!keep_waiting(it, t0, abort, dev_err)) return -1;
  }
}

// Tile number i of this CTA, once it is posted; false past the last one (or
// when the wait was given up).
MOE_DEV bool next_tile(const Ctl& ctl, int i, Tile& t, volatile int* abort, unsigned int* dev_err) {
  if (wait_count(&ctl.ready, i, abort, dev_err) < 0) return false;
  t = ctl.tile[i % kPosted];
  return t.prod >= 0;
}

MOE_DEV void tma_load_4d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2,
                              int32_t c3, uint64_t cache_policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "l"(cache_policy)
      : "memory");
}

// A box into this CTA's own shared memory.
MOE_DEV void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// Instruction descriptor of tcgen05.mma.kind::f16: fp16 A and B, each K-major
// or not, fp32 D.
MOE_DEV uint32_t idesc_f16_f32(uint32_t M, uint32_t N, uint32_t a_mn_major, uint32_t b_mn_major) {
  return (1u << 4) | (a_mn_major << 15) | (b_mn_major << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// Whether k block kb of the row tile t of a symmetric operand lies above the
// diagonal, where only its mirror image is stored.
MOE_DEV bool above(int kb, int t) { return kb / (kTile / kBK) > t; }

// The results (and the weights they move) lie in rows of the stack's own
// matrices, so there the box is turned: half of it at a time, 16 rows x 32
// columns in fp32, 16-byte chunk c of row r at chunk c ^ (r % 8) ^ 4 (r / 8),
// free of bank conflicts.  TMEM gives a lane a whole row; after the turn lane
// l holds, for i = 0 and 1, the 8 columns from 8 (l % 4) of row 8 i + l / 4
// (elements 8 i .. 8 i + 7).
//
// Addresses are one XOR and a constant away from three per-lane bases.  The
// empty asm keeps the compiler from holding all of them in registers around
// the loop over tiles.
MOE_DEV uint32_t here(uint32_t base) {
  asm volatile("" : "+r"(base));
  return base;
}

MOE_DEV void st_shared4(uint32_t a, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}

MOE_DEV void ld_shared4(uint32_t a, float& x, float& y, float& z, float& w) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x), "=f"(y), "=f"(z), "=f"(w) : "r"(a) : "memory");
}

// Rows 16 h .. 16 h + 15 of the 32 that the warp holds in TMEM's layout.
MOE_DEV void box_put_half(uint32_t buf, const uint32_t (&v)[32], int h) {
  const uint32_t l = lane_id();
  if ((l >> 4) == h) {
    const uint32_t r = l & 15, x = here(buf + r * 128 + (((r & 7) ^ ((r >> 3) << 2)) << 4));
#pragma unroll
    for (int c = 0; c < 8; ++c)
      st_shared4(x ^ (c << 4), __uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]), __uint_as_float(v[4 * c + 2]),
                 __uint_as_float(v[4 * c + 3]));
  }
}

MOE_DEV uint32_t box_lane(uint32_t buf) {
  const uint32_t l = lane_id();
  return here(buf + (l >> 2) * 128 + (((2 * (l & 3)) ^ (l >> 2)) << 4));
}

MOE_DEV void box_get(uint32_t buf, float (&v)[16]) {
  const uint32_t x = box_lane(buf);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    ld_shared4((x ^ (((k & 1) ^ ((k >> 1) << 2)) << 4)) + (k >> 1) * 1024, v[4 * k], v[4 * k + 1], v[4 * k + 2],
               v[4 * k + 3]);
}

MOE_DEV void box_put(uint32_t buf, const float (&v)[16]) {
  const uint32_t x = box_lane(buf);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    st_shared4((x ^ (((k & 1) ^ ((k >> 1) << 2)) << 4)) + (k >> 1) * 1024, v[4 * k], v[4 * k + 1], v[4 * k + 2],
               v[4 * k + 3]);
}

// The box transposed: lane l holds, for i = 0 and 1, the 8 rows from 8 (l % 2)
// of column 16 i + l / 2.
MOE_DEV void box_get_turned(uint32_t buf, float (&v)[16]) {
  const uint32_t l = lane_id(), c = l >> 1;
  const uint32_t x = here(buf + (l & 1) * 1024 + (((c >> 2) ^ (4 * (l & 1))) << 4) + (c & 3) * 4);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      asm volatile("ld.shared.f32 %0, [%1];"
                   : "=f"(v[8 * i + k])
                   : "r"((x ^ (((4 * i) ^ k) << 4)) + k * 128)
                   : "memory");
}

// What an epilogue warp knows of its tile.
struct EpiTile {
  int mat, step, cur;
  bool late;            // B's diagonal is kept apart
  int row0, col0;       // the warp's first row and column
  int boxes;            // of 32 columns: 2, or 1 in a narrow tile
  uint8_t* own;         // the lane's piece of the first box of lo, or of A's copy
  uint32_t taddr;       // its accumulator
  uint32_t tfull, tphase, tempty;
  uint32_t buf;         // the warp's box (shared memory)
  uint32_t bar, bar_phase;  // and the barrier of loads into it
  volatile int* abort_flag;
  unsigned int* dev_err;
};

// The accumulator is there; false when the wait was given up.
MOE_DEV bool wait_acc(const EpiTile& t) {
  const bool ok = mbar_wait_cluster(t.tfull, t.tphase, t.abort_flag, t.dev_err);
  tc_fence_after_sync();
  return __all_sync(0xffffffffu, ok) != 0;
}

// It has been read: the MMA issuer may use it again.  Relaxed, because the
// values are in registers by then and nothing else is handed over: a release
// waits for the stores before it (1500 cycles).
MOE_DEV void release(const EpiTile& t) {
  tc_fence_before_sync();
  __syncwarp();
  if (lane_id() == 0)
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(t.tempty) : "memory");
}

// The four epilogues, on two boxes of 32 columns (or one), a lane a row.  Each asks for
// what it reads (A, or X) of the first box before it waits for the accumulator
// and of the second before it works on the first.  Little may spill here:
// shared memory leaves the L1 cache 28 KB, so spilled registers come back from
// L2.  For the same reason every load into registers is made without a
// condition: registers written under one stay live around the loop over tiles.

// The second box, for loads that are made whether or not there is one.
MOE_DEV int second(const EpiTile& t) { return t.boxes - 1; }

// A tile whose part for this warp lies outside the matrix.
MOE_DEV bool epilogue_none(const EpiTile& t) {
  const bool ok = wait_acc(t);
  release(t);
  return ok;
}

// Takes box b from TMEM; after the last one the accumulator is free.
MOE_DEV void take(const EpiTile& t, int b, uint32_t (&acc)[32]) {
  tmem_ld_32cols(t.taddr + b * kBox, acc);
  tmem_ld_wait();
  if (b + 1 == t.boxes) release(t);
}

// 32 bytes, a whole sector, as the last to write them left them in L2.  (With
// 16-byte loads of a lane's own row each sector is fetched twice.)
MOE_DEV void load_sector(const void* p, uint32_t* v) {
  asm volatile("ld.relaxed.gpu.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}
MOE_DEV void store_sector(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The box as fp16 to its place in an operand: through the warp's buffer
// (64-byte swizzle: 16-byte chunk c of row r at c ^ ((r / 2) % 4)) and TMA.
MOE_DEV void store_box(const CUtensorMap* map, const EpiTile& t, int b, const uint32_t (&h)[16]) {
  const uint32_t l = lane_id();
  if (l == 0) bulk_wait_group_read0();  // the store before has read the buffer
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(t.buf + l * 64 + ((c ^ ((l >> 1) & 3)) << 4)),
                 "r"(h[4 * c]), "r"(h[4 * c + 1]), "r"(h[4 * c + 2]), "r"(h[4 * c + 3])
                 : "memory");
  fence_proxy_async_smem();
  __syncwarp();
  if (l == 0) {
    tma_store_3d(map, t.buf, t.col0 + b * kBox, t.row0, t.mat);
    bulk_commit_group();
  }
}

// A = X X^T.
MOE_DEV bool epilogue_gram(const NsMaps& maps, const EpiTile& t) {
  if (!wait_acc(t)) return false;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    if (b >= t.boxes) break;
    uint32_t acc[32], h[16];
    take(t, b, acc);
    constexpr float f = 1.f / (kScaleX * kScaleX);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      h[j] = pack_half2(__uint_as_float(acc[2 * j]) * f, __uint_as_float(acc[2 * j + 1]) * f);
    store_box(&maps.boxA, t, b, h);
    store_sector(t.own + b * kBoxA, h);
    store_sector(t.own + b * kBoxA + 1024, h + 8);
  }
  return true;
}

// B = b A + c A A.
MOE_DEV bool epilogue_poly(const NsMaps& maps, const GemmArgs& p, const EpiTile& t) {
  const uint32_t l = lane_id();
  uint32_t a[2][16];
  load_sector(t.own, a[0]);
  load_sector(t.own + 1024, a[0] + 8);
  const float cb = p.coeff[t.step][1], cc = p.coeff[t.step][2];
  if (!wait_acc(t)) return false;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    if (b >= t.boxes) break;
    uint32_t acc[32], h[16];
    take(t, b, acc);
    if (b == 0) {
      load_sector(t.own + second(t) * kBoxA, a[1]);
      load_sector(t.own + second(t) * kBoxA + 1024, a[1] + 8);
    }
    const bool diagonal = t.late && t.row0 == t.col0 + b * kBox;
    float mine = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 x = unpack_half2(a[b][j]);
      float u = fmaf(cc, __uint_as_float(acc[2 * j]), cb * x.x);
      float v = fmaf(cc, __uint_as_float(acc[2 * j + 1]), cb * x.y);
      if (diagonal) {
        if (l == 2 * j) mine = u, u = 0.f;
        if (l == 2 * j + 1) mine = v, v = 0.f;
      }
      h[j] = pack_half2(u, v);
    }
    if (diagonal) p.diag[static_cast<size_t>(t.mat) * p.mp + t.row0 + l] = mine;
    store_box(&maps.boxB, t, b, h);
  }
  return true;
}

// a plus, where it is kept apart, B's diagonal, for the lane's row.
MOE_DEV float row_factor(const GemmArgs& p, const EpiTile& t) {
  const float d = __ldcg(p.diag + static_cast<size_t>(t.mat) * p.mp + t.row0 + lane_id());
  return p.coeff[t.step][0] + (t.late ? d : 0.f);
}

// The lane's 32 columns of hi, straight from its row.
MOE_DEV void load_row(const __half* p, uint32_t (&h)[16]) {
  load_sector(p, h);
  load_sector(p + 16, h + 8);
}

MOE_DEV const __half* row_of(const GemmArgs& p, const EpiTile& t) {
  return p.hi[t.cur] + (static_cast<size_t>(t.mat) * p.mp + t.row0 + lane_id()) * p.np + t.col0;
}

// hi of the first box comes by TMA into the warp's buffer, hi of the second
// straight into registers (there is no shared memory for a second buffer);
// both are in L2, as operands.
MOE_DEV void ask_hi(const NsMaps& maps, const GemmArgs& p, const EpiTile& t, uint32_t (&other)[16]) {
  if (lane_id() == 0) {
    mbar_arrive_expect_tx(t.bar, kWarpStage);
    tma_load_3d(t.buf, &maps.boxX[t.cur], t.bar, t.col0, t.row0, t.mat);
  }
  load_row(row_of(p, t) + second(t) * kBox, other);
}

// The accumulator and the first box; false when the wait was given up (the
// copy has landed then too).
MOE_DEV bool wait_acc_hi(EpiTile& t, uint32_t (&first)[16]) {
  const uint32_t l = lane_id();
  const bool ok = wait_acc(t);
  volatile int local_abort = 0;
  mbar_wait(t.bar, t.bar_phase, &local_abort, t.dev_err);
  t.bar_phase ^= 1u;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(first[4 * c]), "=r"(first[4 * c + 1]), "=r"(first[4 * c + 2]), "=r"(first[4 * c + 3])
                 : "r"(t.buf + l * 64 + ((c ^ ((l >> 1) & 3)) << 4))
                 : "memory");
  return ok;
}

// X <- a X + B X.
MOE_DEV bool epilogue_apply(const NsMaps& maps, const GemmArgs& p, EpiTile& t) {
  uint32_t hi[2][16], lo[2][8];
  ask_hi(maps, p, t, hi[1]);
  load_sector(t.own, lo[0]);
  load_sector(t.own + second(t) * kBoxX, lo[1]);
  const float f = row_factor(p, t);
  if (!wait_acc_hi(t, hi[0])) return false;
  const bool keep_lo = t.step + 2 < p.steps;  // the last step's X has none
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    if (b >= t.boxes) break;
    uint32_t acc[32];
    take(t, b, acc);
    uint32_t(&h)[16] = hi[b];
    uint32_t n[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float x[4];
      unpack_hi_lo4(h[2 * k], h[2 * k + 1], lo[b][k], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = fmaf(f, x[j], __uint_as_float(acc[4 * k + j]));
      h[2 * k] = pack_half2(x[0], x[1]);
      h[2 * k + 1] = pack_half2(x[2], x[3]);
      n[k] = pack_lo2(x[0], x[1], h[2 * k]) | (pack_lo2(x[2], x[3], h[2 * k + 1]) << 16);
    }
    store_box(&maps.boxX[t.cur ^ 1], t, b, h);
    if (keep_lo) store_sector(t.own + b * kBoxX, n);
  }
  return true;
}

// Eight consecutive bf16 weights (stop of them inside the row), packed.
MOE_DEV void load_bf16(const void* base, size_t el, int stop, bool vec, uint32_t (&w)[4]) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + el;
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = 0;
  if (vec) {
    if (stop > 0) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < stop) w[k / 2] |= static_cast<uint32_t>(__ldcs(p + k)) << (16 * (k & 1));
  }
}

MOE_DEV void store_bf16(void* base, size_t el, int stop, bool vec, const float* v) {
  uint16_t* p = static_cast<uint16_t*>(base) + el;
  if (vec) {
    if (stop > 0)
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < stop) p[k] = static_cast<uint16_t>(pack_bf16x2(v[k], 0.f));
  }
}

// Moves eight consecutive fp32 weights (stop of them inside the row) by o and
// leaves them in o.  (One by one, a step of 24 matrices of 768 x 1536 takes 583
// us instead of 529.  With bf16 weights, which are 113 MB less to move, the
// few registers that this needs cost 3 us of 495.)
MOE_DEV void move_f32(float* d, int stop, bool vec, const NsOutput& out, float* o) {
  if (vec) {
    if (stop > 0) {
      float4* q = reinterpret_cast<float4*>(d);
      const float4 a = __ldcs(q), b = __ldcs(q + 1);
      const float old[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = fmaf(old[k], out.keep, -out.step * o[k]);
      q[0] = make_float4(o[0], o[1], o[2], o[3]);
      q[1] = make_float4(o[4], o[5], o[6], o[7]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < stop) d[k] = o[k] = fmaf(d[k], out.keep, -out.step * o[k]);
  }
}

// The last product: o is the result, or moves the weights, in runs of 8
// elements of the stack's own rows.
MOE_DEV bool epilogue_last(const NsMaps& maps, const GemmArgs& p, const NsStacks& st, EpiTile& t) {
  const uint32_t l = lane_id();
  uint32_t hi[2][16];
  ask_hi(maps, p, t, hi[1]);
  const float f = row_factor(p, t);
  const NsStack& s = st.s[stack_of(st, t.mat)];
  const size_t base = static_cast<size_t>(t.mat - s.first) * p.m * p.n;
  const int rows = s.tall ? p.n : p.m, cols = s.tall ? p.m : p.n;  // the stack's own
  const bool vec = cols % 8 == 0;                                  // runs start on 16 bytes and end inside
  if (!wait_acc_hi(t, hi[0])) return false;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    if (b >= t.boxes) break;
    uint32_t acc[32];
    take(t, b, acc);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 x = unpack_half2(hi[b][j]);
      acc[2 * j] = __float_as_uint(fmaf(f, x.x, __uint_as_float(acc[2 * j])));
      acc[2 * j + 1] = __float_as_uint(fmaf(f, x.y, __uint_as_float(acc[2 * j + 1])));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // the lane's two runs in the stack's own matrix
      const int r0 = s.tall ? t.col0 + b * kBox + (l >> 1) : t.row0 + 16 * h + (l >> 2);
      const int c0 = s.tall ? t.row0 + 16 * h + 8 * (l & 1) : t.col0 + b * kBox + 8 * (l & 3);
      const int rstep = s.tall ? 16 : 8;
      uint32_t w[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int stop = r0 + rstep * i < rows && p.out.kind == kNsWeightBf16 ? min(8, cols - c0) : 0;
        load_bf16(s.weight, base + static_cast<size_t>(r0 + rstep * i) * cols + c0, stop, vec, w[i]);
      }
      float v[16];
      __syncwarp();
      box_put_half(t.buf, acc, h);
      __syncwarp();
      box_get(t.buf, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] *= 1.f / kScaleX;
      if (s.tall) {
        __syncwarp();
        box_put(t.buf, v);
        __syncwarp();
        box_get_turned(t.buf, v);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const size_t at = base + static_cast<size_t>(r0 + rstep * i) * cols + c0;
        const int stop = r0 + rstep * i < rows ? min(8, cols - c0) : 0;
        float* o = v + 8 * i;
        if (p.out.kind == kNsWeightF32) {
          move_f32(static_cast<float*>(s.weight) + at, stop, vec, p.out, o);
          if (s.weight_bf16 != nullptr) store_bf16(s.weight_bf16, at, stop, vec, o);
        } else {
          if (p.out.kind == kNsWeightBf16) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              o[k] = fmaf(k & 1 ? bf16_hi(w[i][k / 2]) : bf16_lo(w[i][k / 2]), p.out.keep, -p.out.step * o[k]);
          }
          store_bf16(s.weight, at, stop, vec, o);
        }
      }
    }
  }
  // the next tile's hi comes into the buffer by TMA (a __syncwarp follows)
  fence_proxy_async_smem();
  return true;
}

__global__ void __launch_bounds__(kThreads, 1)
    ns_products_kernel(const __grid_constant__ NsMaps maps, const __grid_constant__ GemmArgs p,
                       const __grid_constant__ NsStacks st, unsigned int* const dev_err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t smem_base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(cluster_id_x()), npairs = static_cast<int>(num_clusters_x());

  if (warp == 0 && lane == 0) {
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
    ctl.ready = 0;
    ctl.counted = 0;
    for (int w = 0; w < kEpiWarps; ++w) {
      ctl.written[w] = 0;
      mbar_init(smem_u32(&ctl.box[w]), 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&ctl.tmem_base), kTmemCols);
    tmem_relinquish_pair();
    tc_fence_before_sync();
  }
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
      Tile t;
      for (int i = 0; ok && next_tile(ctl, i, t, abort_flag, dev_err); ++i) {
        const int kind = t.prod % 3, cur = (t.prod / 3) & 1;
        asm volatile("fence.proxy.async.global;" ::: "memory");
        const CUtensorMap* mp = kind == kGram ? &maps.X[cur] : kind == kPoly ? &maps.A : &maps.B;
        const CUtensorMap* mq = kind == kPoly ? &maps.A : &maps.X[cur];
        const int nkb = ((kind == kGram ? p.np : p.mp) + kBK - 1) / kBK;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_cluster(smem_u32(&ctl.empty[stage]), phase ^ 1u, abort_flag, dev_err)) {
            ok = false;
            break;
          }
          const uint32_t bar = map_to_cta(smem_u32(&ctl.full[stage]), 0);
          const uint32_t sp = smem_base + stage * kStageBytes, sq = sp + kOperandBytes;
          // both CTAs' boxes count in full, rows and k past the matrix are zeros
          if (leader) mbar_arrive_expect_tx(smem_u32(&ctl.full[stage]), 2 * kStageBytes);
          // 128 rows of the operand and 128 k, or the mirror image of that
          if (kind != kGram && above(kb, t.ti))
            tma_load_4d_pair(sp, mp, bar, 0, kb * kBK, t.ti * (kTile / 64) + 2 * rank, t.mat, policy);
          else
            tma_load_4d_pair(sp, mp, bar, 0, t.ti * kTile + 128 * rank, kb * (kBK / 64), t.mat, policy);
          if (kind == kApply || (kind == kPoly && above(kb, t.tj * p.tn / kTile)))
            tma_load_4d_pair(sq, mq, bar, 0, kb * kBK, (t.tj * p.tn + p.tn / 2 * rank) / 64, t.mat, policy);
          else
            tma_load_4d_pair(sq, mq, bar, 0, t.tj * p.tn + p.tn / 2 * rank, kb * (kBK / 64), t.mat, policy);
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (*abort_flag && leader) {
        // Let the copies already in flight land before the CTA exits.
        for (int k = 0; k < kStages && k < issued; ++k) {
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
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      Tile t;
      for (int i = 0; ok && next_tile(ctl, i, t, abort_flag, dev_err); ++i) {
        const int buf = i & 1;
        if (!mbar_wait_cluster(smem_u32(&ctl.tempty[buf]), ((i >> 1) & 1) ^ 1u, abort_flag, dev_err)) break;
        tc_fence_after_sync();
        const int kind = t.prod % 3;
        const int K = kind == kGram ? p.np : p.mp;
        const int nkb = (K + kBK - 1) / kBK;
        const uint32_t d = tmem_base + buf * kTile;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_cluster(smem_u32(&ctl.full[stage]), phase, abort_flag, dev_err)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sp = smem_base + stage * kStageBytes, sq = sp + kOperandBytes;
          const bool m_major = kind != kGram && above(kb, t.ti);
          const bool n_major = kind == kApply || (kind == kPoly && above(kb, t.tj * p.tn / kTile));
          const uint32_t idesc = idesc_f16_f32(kTile, p.tn, m_major, n_major);
          const int slices = K - kb * kBK >= kBK ? kBK / 16 : 4;  // K is a multiple of 64
          // 16-byte steps from one 16-deep slice to the next: K-major 32 bytes
          // in an atom, then the next atom; else 16 k rows
          const uint64_t pd = smem_desc_sw128(sp, m_major ? kAtomBytes : 16, 1024);
          const uint64_t qd = smem_desc_sw128(sq, n_major ? kAtomBytes : 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            if (kk >= slices) break;
            const uint32_t k_step = (kk >> 2) * (kAtomBytes / 16) + (kk & 3) * 2, mn_step = kk * (2048 / 16);
            umma_bf16_pair(d, pd + (m_major ? mn_step : k_step), qd + (n_major ? mn_step : k_step), idesc,
                           (kb | kk) != 0 ? 1u : 0u);
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
      // All MMAs issued by this thread are complete once `drain` flips.
      umma_commit_pair(smem_u32(&ctl.drain), 0x1);
      volatile int local_abort = 0;
      mbar_wait_cluster(smem_u32(&ctl.drain), 0, &local_abort, dev_err);
    }
    __syncwarp();
  } else if (warp == 2 + kEpiWarps) {
    // ===================== completion (both CTAs) =====================
    // Once the epilogue warps have issued a tile's stores, waits until these
    // are in memory and counts the tile: 2000 to 5000 cycles that the
    // epilogue warps spend on the next tile.  Where there is no next tile to
    // speak of they count their own parts, which is sooner (3 x 1001 x 363:
    // 177 -> 163 us; a step of 24 matrices of 768 x 1536: 490 -> 512 us).
    //
    // Each lane waits for one epilogue warp, and lane 0 alone fences, counts
    // and gives the tile's place back.  So what the other lanes have acquired,
    // and their reading of the place, are ordered before it by a __syncwarp
    // (votes and shuffles order no memory), and all lanes leave together.
    int upto = 0;
    Tile t;
    for (int i = 0;; ++i) {
      const bool got = next_tile(ctl, i, t, abort_flag, dev_err);
      if (!__all_sync(0xffffffffu, got)) break;
      bool fresh = false;  // newly seen stores to fence
      if (i >= upto) {     // all that every warp has issued by now, with one fence
        int v = lane < kEpiWarps ? wait_count(&ctl.written[lane], i, abort_flag, dev_err) : 0x7fffffff;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (v < 0) break;
        upto = v;
        fresh = true;
      }
      __syncwarp();
      if (lane == 0) {
        if (!p.direct) {
          if (fresh) {
            asm volatile("fence.proxy.async.global;" ::: "memory");
            __threadfence();
          }
          if (t.prod + 1 < 3 * p.steps) count_done(p, t);
        }
        count_store(&ctl.counted, i + 1);
      }
    }
    __syncwarp();
  } else if (warp == 3 + kEpiWarps) {
    // ===================== next tiles (both CTAs) =====================
    // The CTA's tiles in order, each posted when the product that it reads is
    // complete, at most kPosted ahead of the last one that is done with.  The
    // others would each spend 500 to 1500 cycles a tile on finding it and on
    // the round trip to the counter, the producer in the middle of its loads.
    if (lane == 0) {
      Walk w;
      int i = 0;
      bool ok = true;
      for (int idx = pair; ok && w.to(p, idx); idx += npairs, ++i) {
        ok = wait_count(&ctl.counted, i - kPosted, abort_flag, dev_err) >= 0 &&
             wait_product(p, w.prod, w.mat, abort_flag, dev_err);
        if (!ok) break;
        ctl.tile[i % kPosted] = Tile{w.prod, w.mat, w.ti, w.tj};
        count_store(&ctl.ready, i + 1);
      }
      if (ok && wait_count(&ctl.counted, i - kPosted, abort_flag, dev_err) >= 0) {
        ctl.tile[i % kPosted].prod = -1;
        count_store(&ctl.ready, i + 1);
      }
    }
    __syncwarp();
  } else {
    // ===================== epilogue (both CTAs) =====================
    // Warp w: TMEM lanes 32 (w % 4) .. + 31 and columns 64 ((w - 2) / 4) ..
    // + 63, in two boxes of 32 columns.
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t tempty0 = map_to_cta(smem_u32(&ctl.tempty[0]), 0);
    const uint32_t tempty1 = map_to_cta(smem_u32(&ctl.tempty[1]), 0);
    const uint32_t box = smem_base + kStages * kStageBytes + (warp - 2) * kWarpStage;
    uint32_t bar_phase = 0;
    Tile t;
    for (int i = 0;; ++i) {
      bool got = next_tile(ctl, i, t, abort_flag, dev_err);
      if (!__all_sync(0xffffffffu, got)) break;
      const int kind = t.prod % 3, step = t.prod / 3, buf = i & 1;
      EpiTile e;
      e.mat = t.mat, e.step = step, e.cur = step & 1;
      e.late = step + 2 >= p.steps;
      e.row0 = t.ti * kTile + 128 * static_cast<int>(rank) + q * 32;
      e.col0 = t.tj * p.tn + part * (p.tn / 4);
      e.boxes = p.tn / 128;
      const int ncols = kind == kApply ? p.np : p.mp;
      e.own = (kind == kApply ? p.lo : p.a) + lane * 32 +
              box_number(t.mat, p.mp, ncols, e.row0, e.col0) * (kind == kApply ? kBoxX : kBoxA);
      e.taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kTile + part * (p.tn / 4);
      e.tfull = smem_u32(&ctl.tfull[buf]);
      e.tphase = (i >> 1) & 1;
      e.tempty = buf ? tempty1 : tempty0;
      e.buf = box;
      e.bar = smem_u32(&ctl.box[warp - 2]), e.bar_phase = bar_phase;
      e.abort_flag = abort_flag;
      e.dev_err = dev_err;
      // padded sizes are multiples of 64: the warp's part is inside or outside
      if (e.row0 >= p.mp || e.col0 >= ncols)
        got = epilogue_none(e);
      else if (kind == kGram)
        got = epilogue_gram(maps, e);
      else if (kind == kPoly)
        got = epilogue_poly(maps, p, e);
      else if (step + 1 < p.steps)
        got = epilogue_apply(maps, p, e);
      else
        got = epilogue_last(maps, p, st, e);
      bar_phase = e.bar_phase;
      if (!got) break;
      __syncwarp();
      if (lane == 0) {
        bulk_wait_group0();  // TMA stores are complete for their own thread only
        if (p.direct && t.prod + 1 < 3 * p.steps) {
          asm volatile("fence.proxy.async.global;" ::: "memory");
          count_done(p, t);
        }
      }
      if (lane == 0) count_store(&ctl.written[warp - 2], i + 1);
    }
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
  float *partial, *diag;
  unsigned int* done;
  __half *hi[2], *A, *B;
  uint8_t *lo, *a;
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
  const size_t x = static_cast<size_t>(count) * mp * np, a = static_cast<size_t>(count) * mp * mp * 2;
  w.partial = reinterpret_cast<float*>(take(static_cast<size_t>(count) * kNormChunks * 4));
  w.done = reinterpret_cast<unsigned int*>(take(static_cast<size_t>(count) * 3 * MOE_MAX_NS_STEPS * 4));
  w.diag = reinterpret_cast<float*>(take(static_cast<size_t>(count) * mp * 4));
  for (int i = 0; i < 2; ++i) w.hi[i] = reinterpret_cast<__half*>(take(2 * x));
  w.lo = reinterpret_cast<uint8_t*>(take(x));
  w.a = reinterpret_cast<uint8_t*>(take(a));
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
    const void* fn = reinterpret_cast<const void*>(ns_products_kernel);
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
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
    e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
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

// [count, rows, cols] fp16 in 32 x 32 boxes with the 64-byte swizzle.
cudaError_t box_map(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* p, int count, int rows,
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

// Norms, then X_0.  (In batches of what the L2 cache holds of g and m, so that
// the second pass finds them there a step of 24 matrices of 768 x 1536 took 6
// us longer.)
template <typename GT, int VEC>
cudaError_t launch_first(const NsProblem& pr, const Buffers& w, int mp, int np, cudaStream_t s) {
  const size_t elems = static_cast<size_t>(pr.m) * pr.n;
  size_t chunk = (elems + kNormChunks - 1) / kNormChunks;
  chunk = std::max<size_t>((chunk + 3) / 4 * 4, 8192);
  const int chunks = static_cast<int>((elems + chunk - 1) / chunk);
  cudaError_t e = launch_kernel(ns_norm_kernel<GT, VEC>, dim3(chunks, pr.count), dim3(kNormThreads), 0, s, false,
                                pr.stacks, pr.momentum, pr.nesterov, elems, chunk, w.partial, w.done, 3 * pr.steps);
  if (e != cudaSuccess) return e;
  return launch_kernel(ns_load_kernel<GT, VEC>, dim3((mp / 64) * (np / 64), pr.count), dim3(256), 0, s, true,
                       pr.stacks, pr.momentum, pr.nesterov, pr.m, pr.n, mp, np, chunks, pr.eps,
                       static_cast<const float*>(w.partial), w.hi[0], w.lo);
}

}  // namespace

size_t ns_workspace_bytes(int count, int m, int n) { return carve(nullptr, count, pad64(m), pad64(n)).bytes; }

cudaError_t launch_newton_schulz(const NsProblem& pr, void* workspace, cudaStream_t s) {
  if (ns_small_fits(pr.m, pr.n)) return launch_ns_small(pr, s);
  PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  int pairs = 0;
  unsigned int* err = nullptr;
  cudaError_t e = setup(&enc, &pairs);
  if (e != cudaSuccess) return e;
  if ((e = device_error_address(&err)) != cudaSuccess) return e;
  const int mp = pad64(pr.m), np = pad64(pr.n), count = pr.count;
  const Buffers w = carve(workspace, count, mp, np);

  // four values at a time where rows (of either orientation) start on a multiple of four
  const bool vec = pr.m % 4 == 0 && pr.n % 4 == 0;
  if (pr.grad_fp32)
    e = vec ? launch_first<float, 4>(pr, w, mp, np, s) : launch_first<float, 1>(pr, w, mp, np, s);
  else
    e = vec ? launch_first<uint16_t, 4>(pr, w, mp, np, s) : launch_first<uint16_t, 1>(pr, w, mp, np, s);
  if (e != cudaSuccess) return e;

  NsMaps maps;
  for (int i = 0; i < 2; ++i)
    if ((e = operand_map(enc, &maps.X[i], w.hi[i], count, mp, np)) != cudaSuccess ||
        (e = box_map(enc, &maps.boxX[i], w.hi[i], count, mp, np)) != cudaSuccess)
      return e;
  if ((e = box_map(enc, &maps.boxA, w.A, count, mp, mp)) != cudaSuccess) return e;
  if ((e = box_map(enc, &maps.boxB, w.B, count, mp, mp)) != cudaSuccess) return e;
  if ((e = operand_map(enc, &maps.A, w.A, count, mp, mp)) != cudaSuccess) return e;
  if ((e = operand_map(enc, &maps.B, w.B, count, mp, mp)) != cudaSuccess) return e;

  GemmArgs a{};
  a.mp = mp, a.np = np, a.m = pr.m, a.n = pr.n;
  a.steps = pr.steps;
  // Narrow tiles while one wave of them holds the widest product, two with a
  // short k: what counts then is how long a tile takes, and not that operands
  // are loaded twice as often.  3 x 1001 x 363: 163 -> 133 us.  Between one and
  // two waves, wide / narrow: 12 x 256 x 1024 132 / 119, 12 x 512 x 512 139 /
  // 127, 4 x 512 x 2048 175 / 164, 3 x 640 x 1280 156 / 141, 3 x 768 x 1536
  // 173 / 162, 4 x 768 x 1536 (1.9 waves) 184 / 185; where 1.9 waves of narrow
  // ones are one of wide ones they lose (18 x 512 x 512 147 / 161, 8 x 768 x 768
  // 166 / 173).  Past 768 rows there is little to gain and more to lose: 3 x 832
  // x 832 156 / 146, 3 x 1024 x 1024 174 / 170, 2 x 1280 x 1280 190 / 193, 3 x
  // 1280 x 1280 212 / 211, 2 x 1536 x 1536 227 / 228, 1 x 2048 x 2048 251 / 280.
  // Past two waves 30 x 256 x 1024 (3.2) takes 153 / 160.
  a.tn = 128;
  if (static_cast<long>(count) * Walk::tiles(a, kApply) > (mp <= 3 * kTile ? 2 : 1) * pairs) a.tn = kTile;
  a.direct = static_cast<long>(count) * Walk::tiles(a, kGram) <= pairs;
  a.count = count;
  // Groups whose smallest product has two tiles for each pair, so that the way
  // from one product to the next is covered, and no more, so that X may still
  // be in L2 for its second reading: 12 matrices of 2048 x 8192 four at a time
  // 5.36 ms, all at once 5.68, two at a time 5.66.  For 192 of 768 x 1536 any
  // size from 24 on is the same.
  const int groups = std::max(1, count / std::max(1, 2 * pairs / Walk::tiles(a, kGram)));
  a.group = (count + groups - 1) / groups;
  for (int k = 0; k < pr.steps; ++k)
    for (int j = 0; j < 3; ++j) a.coeff[k][j] = pr.coeff[k][j];
  for (int i = 0; i < 2; ++i) a.hi[i] = w.hi[i];
  a.lo = w.lo, a.a = w.a;
  a.diag = w.diag;
  a.done = w.done;
  a.out = pr.out;
  // more pairs than the widest product has tiles would find nothing to do
  const long most = static_cast<long>(count) * std::max(Walk::tiles(a, kApply), Walk::tiles(a, kGram));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<long>(pairs, most)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, ns_products_kernel, maps, a, pr.stacks, err);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
