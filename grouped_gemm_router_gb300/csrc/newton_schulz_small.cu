// Newton-Schulz for matrices of at most 128 rows (short side) and 2048
// columns, all steps on chip: one CTA for each 256 columns, a cluster of up
// to eight CTAs for a matrix, one launch for everything.
//
// The three products of a step depend on one another, and on matrices this
// small each takes well under a microsecond: what counts is the way from one
// to the next.  Through memory and a counter 4 matrices of 128 x 256 take
// 82 us for five steps (the tiled kernel of newton_schulz.cu); here X, A and B
// stay in shared memory and TMEM, and they take 30 us.
//
//   TMEM (512 columns): X in fp32 (256), A = X X^T (128), A A (128)
//   shared memory: X in fp16 (64 KB), A and then B in fp16 (32 KB), A's
//   partial sums for the cluster (64 KB); at the start and the end an fp32
//   stash of the CTA's columns
//
// X lives in TMEM in fp32 as the accumulator of the product B X: scaled by a
// in place, it is the linear term of the next X, and the product adds to it.
// So the linear term is exact to fp32 (newton_schulz.cu explains why it has
// to be kept apart), and in the last two steps B's diagonal joins the scale.
// A's products are fp16 with fp32 sums.
//
// With several CTAs, each has the product of its columns; these are added in
// rank order, each CTA a part of the rows, and handed to all in fp16.
#include <cuda_fp16.h>

#include <algorithm>

#include "moe_device.cuh"
#include "moe_kernels.cuh"
#include "newton_schulz_parts.cuh"

namespace moe {

namespace {

constexpr int kWarps = kThreads / 32;
constexpr int kBlockBytes = kRowsMax * 64 * 2;   // 128 rows x 64 columns of fp16
constexpr int kXBytes = kSlice / 64 * kBlockBytes;
constexpr int kABytes = 2 * kBlockBytes;
constexpr int kPartBytes = kRowsMax * 128 * 4;
constexpr int kStashBytes = kRowsMax * kPitch * 4;
constexpr int kSmemBytes = kXBytes + (kStashBytes > kABytes + kPartBytes ? kStashBytes : kABytes + kPartBytes) + 1024;
constexpr uint32_t kTmemX = 0, kTmemA = 256, kTmemP = 384;
constexpr float kScaleX = 4096.f;                // as in newton_schulz.cu

struct SmallArgs {
  int count, m, n;
  int slice;        // columns of a CTA, a multiple of 64
  int steps;
  float coeff[MOE_MAX_NS_STEPS][3];
  float mu, eps;
  int nesterov;
  NsOutput out;
};

struct Ctl {
  uint64_t done;                    // the products issued so far are complete
  uint32_t tmem_base;
  int abort;
  float red[kWarps];
  float sums[kMaxCluster];          // the CTAs' sums of squares
  float diag[kRowsMax];
};

MOE_DEV int stack_of(const NsStacks& st, int mat) {
  int s = 0;
  while (s + 1 < st.n && mat >= st.s[s + 1].first) ++s;
  return s;
}

MOE_DEV uint32_t pack_half2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Stores 32 columns of the executing warp's lanes into TMEM.
MOE_DEV void tmem_st_32cols(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

MOE_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// fp16 A (K-major) and B (K-major or N-major), fp32 D, M = 128.
MOE_DEV uint32_t idesc_f16(uint32_t N, uint32_t b_mn_major) {
  return (1u << 4) | (b_mn_major << 16) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}

// 16-byte chunk c (8 fp16 columns) of row r in a K-major operand of 64-column
// blocks of 128 rows with the 128-byte swizzle.
MOE_DEV uint32_t chunk_at(uint32_t base, uint32_t r, uint32_t c) {
  return base + (c >> 3) * kBlockBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

MOE_DEV void st_shared_u4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Columns [col, col + 32) of row r as fp16 into an operand.
MOE_DEV void put_halves(uint32_t base, uint32_t r, uint32_t col, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    st_shared_u4(chunk_at(base, r, col / 8 + c), pack_half2(v[8 * c], v[8 * c + 1]), pack_half2(v[8 * c + 2], v[8 * c + 3]),
                 pack_half2(v[8 * c + 4], v[8 * c + 5]), pack_half2(v[8 * c + 6], v[8 * c + 7]));
}

MOE_DEV void get_acc(uint32_t taddr, float (&v)[32]) {
  uint32_t u[32];
  tmem_ld_32cols(taddr, u);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
}

MOE_DEV void put_acc(uint32_t taddr, const float (&v)[32]) {
  uint32_t u[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(v[j]);
  tmem_st_32cols(taddr, u);
}

// Generic writes to shared memory and TMEM accesses of all threads before
// what one thread issues to the tensor core after.
MOE_DEV void hand_to_mma() {
  fence_proxy_async_smem();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
}

// VEC consecutive elements.
template <int VEC>
MOE_DEV void load_run(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  } else {
    v[0] = *p;
  }
}
template <int VEC>
MOE_DEV void load_run(const uint16_t* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
  } else {
    v[0] = bf16_lo(*p);
  }
}
template <int VEC>
MOE_DEV void store_run(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *p = v[0];
}
template <int VEC>
MOE_DEV void store_run(uint16_t* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  else
    *p = static_cast<uint16_t>(pack_bf16x2(v[0], 0.f));
}

// Visits the part's runs, batch(VEC) a thread at a time.
template <int VEC, typename Load, typename Use>
MOE_DEV void visit(const Part& q, Load load, Use use) {
  constexpr int kBatch = batch(VEC);
  const int total = run_count(q);
#pragma unroll 1
  for (int s0 = threadIdx.x; s0 < total; s0 += kThreads * kBatch) {
    int at[kBatch], spot[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      place_run<VEC>(q, s0 + k * kThreads, at[k], spot[k]);
      load(k, at[k]);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (spot[k] >= 0) use(k, spot[k], at[k]);
  }
}

template <int VEC>
MOE_DEV void stash_put(uint32_t stash, int spot, const float (&v)[VEC]) {
  if constexpr (VEC == 4)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stash + spot * 4), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3])
                 : "memory");
  else
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(stash + spot * 4), "f"(v[0]) : "memory");
}
template <int VEC>
MOE_DEV void stash_get(uint32_t stash, int spot, float (&v)[VEC]) {
  if constexpr (VEC == 4)
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(stash + spot * 4)
                 : "memory");
  else
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0]) : "r"(stash + spot * 4) : "memory");
}

// Momentum, and u into the stash; returns the thread's sum of squares.
template <typename GT, int VEC>
MOE_DEV float take_in(const SmallArgs& p, const NsStack& s, size_t base, const Part& q, uint32_t stash) {
  const GT* g = static_cast<const GT*>(s.grad) + base;
  float* mom = s.momentum ? s.momentum + base : nullptr;
  constexpr int kBatch = batch(VEC);
  float sq = 0.f, gv[kBatch][VEC], mv[kBatch][VEC];
  visit<VEC>(
      q,
      [&](int k, int i) {
        load_run<VEC>(g + i, gv[k]);
        if (mom != nullptr) load_run<VEC>(mom + i, mv[k]);
      },
      [&](int k, int spot, int i) {
        if (mom != nullptr) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            mv[k][j] = fmaf(p.mu, mv[k][j], gv[k][j]);
            gv[k][j] = p.nesterov ? fmaf(p.mu, mv[k][j], gv[k][j]) : mv[k][j];
          }
          store_run<VEC>(mom + i, mv[k]);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) sq = fmaf(gv[k][j], gv[k][j], sq);
        stash_put<VEC>(stash, spot, gv[k]);
      });
  return sq;
}

// The result, or the weights it moves, from the stash.
template <int VEC>
MOE_DEV void give_out(const SmallArgs& p, const NsStack& s, size_t base, const Part& q, uint32_t stash) {
  constexpr int kBatch = batch(VEC);
  float w[kBatch][VEC];
  uint16_t* const half = static_cast<uint16_t*>(p.out.kind == kNsWeightF32 ? s.weight_bf16 : s.weight) + base;
  float* const full = static_cast<float*>(s.weight) + base;
  const bool store_half = p.out.kind != kNsWeightF32 || s.weight_bf16 != nullptr;
  visit<VEC>(
      q,
      [&](int k, int i) {
        if (p.out.kind == kNsWeightBf16)
          load_run<VEC>(half + i, w[k]);
        else if (p.out.kind == kNsWeightF32)
          load_run<VEC>(full + i, w[k]);
      },
      [&](int k, int spot, int i) {
        float o[VEC];
        stash_get<VEC>(stash, spot, o);
        if (p.out.kind != kNsPlain) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) o[j] = fmaf(w[k][j], p.out.keep, -p.out.step * o[j]);
        }
        if (p.out.kind == kNsWeightF32) store_run<VEC>(full + i, o);
        if (store_half) store_run<VEC>(half + i, o);
      });
}

template <typename GT, int VEC>
__global__ void __launch_bounds__(kThreads, 1)
    ns_small_kernel(const __grid_constant__ SmallArgs p, const __grid_constant__ NsStacks st, unsigned int* const dev_err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t xs = smem_u32(smem), as = xs + kXBytes, part = as + kABytes;
  const uint32_t stash = as;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, cq = warp >> 2;
  const uint32_t row = 32 * q + lane;              // the thread's row of X, A and B
  const uint32_t rank = cluster_ctarank();
  uint32_t ranks;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
  const int mat = blockIdx.x / ranks;
  const NsStack& s = st.s[stack_of(st, mat)];
  const size_t base = static_cast<size_t>(mat - s.first) * p.m * p.n;
  const int c0 = rank * p.slice, width = slice_width(p.n, p.slice, rank);
  volatile int* abort_flag = &ctl.abort;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&ctl.done), 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&ctl.tmem_base), 512);
    tmem_relinquish();
    tc_fence_before_sync();
  }
  cluster_sync_all();  // all CTAs run: their shared memory may be written
  tc_fence_after_sync();
  const uint32_t tmem = ctl.tmem_base + (static_cast<uint32_t>(q * 32) << 16);

  // ---- momentum, u into the stash, its sum of squares ----
  const bool runs = VEC == 4 && !s.tall;
  const Part mine = runs ? part_of<VEC>(false, p.m, p.n, c0, width) : part_of<1>(s.tall, p.m, p.n, c0, width);
  float sq = runs ? take_in<GT, VEC>(p, s, base, mine, stash) : take_in<GT, 1>(p, s, base, mine, stash);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  if (lane == 0) ctl.red[warp] = sq;
  __syncthreads();
  if (threadIdx.x < ranks) {  // this CTA's sum to every CTA
    float t = 0.f;
    for (int w = 0; w < kWarps; ++w) t += ctl.red[w];
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_cta(smem_u32(&ctl.sums[rank]), threadIdx.x)), "f"(t)
                 : "memory");
  }
  cluster_sync_all();
  float total = 0.f;
  for (uint32_t r = 0; r < ranks; ++r) total += ctl.sums[r];
  // as in newton_schulz.cu: no number, or past fp32, makes the matrix NaN
  const float inv = total < INFINITY ? kScaleX / (sqrtf(total) + p.eps) : NAN;

  // ---- X_0: fp32 into TMEM, fp16 into shared memory ----
  const int xcol = cq * 64;  // the warp's columns of X, if the slice has them
  const bool has_x = xcol < p.slice;
  if (has_x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const int c = xcol + 32 * h + j;
        float x[4];
        stash_get<4>(stash, row * kPitch + c, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j + k] = static_cast<int>(row) < p.m && c + k < width ? x[k] * inv : 0.f;
      }
      put_acc(tmem + kTmemX + xcol + 32 * h, v);
      put_halves(xs, row, xcol + 32 * h, v);
    }
    tmem_st_wait();
  }
  hand_to_mma();

  const int kslices = (p.m + 15) / 16;  // k of A and B: rows past the matrix are zeros
  uint32_t phase = 0;
  auto wait_mma = [&]() {
    mbar_wait(smem_u32(&ctl.done), phase, abort_flag, dev_err);
    phase ^= 1u;
    tc_fence_after_sync();
  };
  for (int step = 0; step < p.steps; ++step) {
    const bool late = step + 2 >= p.steps, last = step + 1 == p.steps;
    const float ca = p.coeff[step][0], cb = p.coeff[step][1], cc = p.coeff[step][2];
    // ---- A = X X^T (this CTA's columns) ----
    if (threadIdx.x == 0) {
      const uint32_t idesc = idesc_f16(128, 0);
      for (int k = 0; k < p.slice / 16; ++k) {
        const uint64_t d = smem_desc_sw128(xs + (k >> 2) * kBlockBytes + (k & 3) * 32, 16, 1024);
        umma_bf16(ctl.tmem_base + kTmemA, d, d, idesc, k > 0);
      }
      umma_commit(smem_u32(&ctl.done));
    }
    if (!late && has_x) {  // meanwhile the linear term
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        get_acc(tmem + kTmemX + xcol + 32 * h, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= ca;
        put_acc(tmem + kTmemX + xcol + 32 * h, v);
      }
      tmem_st_wait();
    }
    wait_mma();
    float a[32];  // A's columns 32 cq .. of the thread's row
    get_acc(tmem + kTmemA + 32 * cq, a);
#pragma unroll
    for (int j = 0; j < 32; ++j) a[j] *= 1.f / (kScaleX * kScaleX);
    if (ranks == 1) {
      put_halves(as, row, 32 * cq, a);
    } else {
      // partial sums into this CTA's memory (16-byte chunk c of row r at c ^
      // (r % 8)), then each CTA adds a part of the rows and hands it to all:
      // 9000 cycles with eight CTAs (10300 when the sums' owners were sent
      // the parts instead of fetching them)
#pragma unroll
      for (int c = 0; c < 8; ++c)
        st_shared_u4(part + row * 512 + (((8 * cq + c) ^ (row & 7)) << 4), __float_as_uint(a[4 * c]),
                     __float_as_uint(a[4 * c + 1]), __float_as_uint(a[4 * c + 2]), __float_as_uint(a[4 * c + 3]));
      cluster_sync_all();
      const uint32_t rows = kRowsMax / ranks;
      for (uint32_t i = threadIdx.x; i < rows * 32; i += kThreads) {
        const uint32_t r = rank * rows + (i >> 5), c4 = i & 31;
        const uint32_t from = part + r * 512 + ((c4 ^ (r & 7)) << 4);
        float x[kMaxCluster][4];
#pragma unroll
        for (uint32_t k = 0; k < kMaxCluster; ++k)
          if (k < ranks)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[k][0]), "=f"(x[k][1]), "=f"(x[k][2]), "=f"(x[k][3])
                         : "r"(map_to_cta(from, k)));
#pragma unroll
        for (uint32_t k = 1; k < kMaxCluster; ++k)
          if (k < ranks)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[0][j] += x[k][j];
        const uint32_t h0 = pack_half2(x[0][0], x[0][1]), h1 = pack_half2(x[0][2], x[0][3]);
        const uint32_t to = chunk_at(as, r, c4 >> 1) + (c4 & 1) * 8;
#pragma unroll
        for (uint32_t k = 0; k < kMaxCluster; ++k)
          if (k < ranks)
            asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(map_to_cta(to, k)), "r"(h0), "r"(h1)
                         : "memory");
      }
      asm volatile("fence.proxy.async;" ::: "memory");
      cluster_sync_all();
    }
    hand_to_mma();
    // ---- A A ----
    if (threadIdx.x == 0) {
      const uint32_t idesc = idesc_f16(128, 0);
      for (int k = 0; k < kslices; ++k) {
        const uint64_t d = smem_desc_sw128(as + (k >> 2) * kBlockBytes + (k & 3) * 32, 16, 1024);
        umma_bf16(ctl.tmem_base + kTmemP, d, d, idesc, k > 0);
      }
      umma_commit(smem_u32(&ctl.done));
    }
    // A as the product has it, rounded (and summed over the cluster): B's
    // error from a rounding of A is (b + 2 c A) times it, a cancellation that
    // an unrounded A in b A would lose (3.6e-3 instead of 2.4e-3 off at 65 x 200)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t u[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                   : "r"(chunk_at(as, row, 4 * cq + c))
                   : "memory");
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
        a[8 * c + 2 * j] = f.x, a[8 * c + 2 * j + 1] = f.y;
      }
    }
    wait_mma();
    // ---- B = b A + c A A over A's place ----
    {
      float v[32];
      get_acc(tmem + kTmemP + 32 * cq, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = fmaf(cc, v[j], cb * a[j]);
      if (late && cq == q) {  // the thread's diagonal element is among its columns
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == lane) {
            ctl.diag[row] = v[j];
            v[j] = 0.f;
          }
      }
      put_halves(as, row, 32 * cq, v);
    }
    if (late) {
      __syncthreads();
      if (has_x) {
        const float f = ca + ctl.diag[row];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[32];
          get_acc(tmem + kTmemX + xcol + 32 * h, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= f;
          put_acc(tmem + kTmemX + xcol + 32 * h, v);
        }
        tmem_st_wait();
      }
    }
    hand_to_mma();
    // ---- X <- (scaled X) + B X ----
    if (threadIdx.x == 0) {
      const uint32_t idesc = idesc_f16(p.slice, 1);
      for (int k = 0; k < kslices; ++k)
        umma_bf16(ctl.tmem_base + kTmemX, smem_desc_sw128(as + (k >> 2) * kBlockBytes + (k & 3) * 32, 16, 1024),
                  smem_desc_sw128(xs + k * 2048, kBlockBytes, 1024), idesc, 1u);
      umma_commit(smem_u32(&ctl.done));
    }
    wait_mma();
    if (has_x) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        get_acc(tmem + kTmemX + xcol + 32 * h, v);
        if (!last) {
          put_halves(xs, row, xcol + 32 * h, v);
        } else {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float x[4] = {v[j] * (1.f / kScaleX), v[j + 1] * (1.f / kScaleX), v[j + 2] * (1.f / kScaleX),
                                v[j + 3] * (1.f / kScaleX)};
            stash_put<4>(stash, row * kPitch + xcol + 32 * h + j, x);
          }
        }
      }
    }
    hand_to_mma();
  }

  // ---- the result, or the weights it moves ----
  if (runs)
    give_out<VEC>(p, s, base, mine, stash);
  else
    give_out<1>(p, s, base, mine, stash);
  // no CTA of the cluster leaves while another may read its memory
  tc_fence_before_sync();
  cluster_sync_all();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(ctl.tmem_base, 512);
  }
}

}  // namespace

// Over the whole range this is faster than the tiled kernel, five steps from
// fp32: 1 of 128 x 128 24 us (tiled 77), 2048 of 128 x 256 422 (1634), 16 of
// 128 x 2048 100 (145), 256 of them 893 (990), 64 of 8 x 2048 216 (238).
bool ns_small_fits(int m, int n) { return m <= kRowsMax && n <= kSlice * kMaxCluster; }

cudaError_t launch_ns_small(const NsProblem& pr, cudaStream_t s) {
  unsigned int* err = nullptr;
  cudaError_t e = device_error_address(&err);
  if (e != cudaSuccess) return e;
  const int ranks = cluster_ranks(pr.n);
  SmallArgs a{};
  a.count = pr.count, a.m = pr.m, a.n = pr.n;
  a.slice = slice_columns(pr.n, ranks);
  a.steps = pr.steps;
  for (int k = 0; k < pr.steps; ++k)
    for (int j = 0; j < 3; ++j) a.coeff[k][j] = pr.coeff[k][j];
  a.mu = pr.momentum;
  a.eps = pr.eps;
  a.nesterov = pr.nesterov;
  a.out = pr.out;
  // four elements at a time where rows (of either orientation) start on a multiple of four
  const bool vec = pr.m % 4 == 0 && pr.n % 4 == 0;
  auto kernel = pr.grad_fp32 ? (vec ? ns_small_kernel<float, 4> : ns_small_kernel<float, 1>)
                             : (vec ? ns_small_kernel<uint16_t, 4> : ns_small_kernel<uint16_t, 1>);
  e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pr.count) * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a, pr.stacks, err);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
