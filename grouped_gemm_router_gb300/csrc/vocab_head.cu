// The vocabulary product at the end of a language model, z = x W^T with
// x [T, D] and the table W [V, D] (bf16), under a softmax that is compared with
// one label a token (cross entropy) or with a teacher's K entries a token
// (distillation).  The logits z [T, V] never reach memory.
//
// Forward: with c = log2(e) / temperature, every token needs
//   lse = ln 2 * log2 sum_v 2^(c z_v)
// and z at its targets.  vocab_kernel<kStats> computes 256 x 256 tiles of z on
// CTA pairs (tcgen05.mma.cta_group::2, fp32 in TMEM, long sums in parts: parts_of
// below); its epilogue keeps the running maximum and sum of a row in registers over
// a run of tiles, picks the targets that lie in the tile, and writes one (maximum,
// sum) pair a row and run.  vocab_finish_kernel joins them and writes lse and the
// loss.
//
// Backward, by pieces of the vocabulary:
//   dz_v = a 2^(c z_v - lse / ln 2)  (+ the targets' own terms)
// vocab_kernel<kDz> recomputes z and stores dz of the piece as bf16;
// vocab_kernel<kGrad> runs both products of it in one launch,
//   dx [T, D] += dz W[piece],   dW[piece] = dz^T x,
// so that the tiles of one fill the last wave of the other.  The values at the
// targets (a q - p, where the two terms nearly cancel for a token that is
// known well) are formed in fp32 apart from it: a label's by the epilogue from the
// loss, a teacher's entries' by vocab_distill_targets_kernel, over what the epilogue
// has stored.
// dz is stored block by block of 64 columns, [Vc / 64][T][64], so that a warp's
// 32 x 64 box is 4 KB in a row.  It is the one intermediate that is rounded to fewer
// than 32 bits: a bf16 operand is what the tensor cores take at full rate, and a
// relative rounding of 2^-9 of each term averages out in sums over V or T.
//
// Shared-memory operand layouts (TMA, 128-byte swizzle): x, W and dz are all
// read in boxes {64 columns, 128 rows, 2 column blocks} of the view
// {64, rows, columns / 64}.  Along the reduction such a box is two K-major
// swizzle atoms of 128 rows (slice kk at atom kk / 4, byte 32 (kk % 4)), across
// it 128 M- or N-major columns of 128 k (LBO = one block of 16 KB, slice kk at
// byte 2048 kk), so one tensor map serves every use.  Rows and columns outside
// the tensor read zeros.
#include <algorithm>
#include <mutex>

#include "moe_device.cuh"
#include "moe_kernels.cuh"
#include "vocab_plan.cuh"

namespace moe {
namespace {

constexpr int kStages = 3;
constexpr int kOperandBytes = 128 * kBK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kBoxes = 4;      // 32-column boxes of an epilogue warp
constexpr uint32_t kTmemCols = 512;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.442695040888963407f;

// A warp's buffer for what it stores: 32 rows of 128 bytes, 16-byte chunk c of row r at c ^ (r % 8)
// (TMA's 128-byte swizzle, and free of bank conflicts when a lane has a row).
constexpr int kBoxBytes = 4096;
constexpr int kSmemBytes = kStages * kStageBytes + kEpiWarps * kBoxBytes + 1024;

struct VocabArgs : VocabWork {
  int T, V, D;
  int box;                 // rows of a box of tokens
  int parts;               // sums that a logit is made of
  int v0, Vc, Vcp;         // kDz, kGrad: the piece's first row, its rows, and those rounded up to 64
  float c;
  unsigned int* dev_err;
  // targets: labels (K = 0), or kStats: sorted keys [T, K]
  const void* labels;
  int labels64;
  const uint32_t* keys;
  int K;
  float* target;           // kStats: z at the targets [T] or [T, K]
  float2* part;            // kStats: (maximum, sum) [2 runs, rows_padded]
  int rows_padded;
  const float* row_a;      // kDz, K > 0: a of each row
  const float* lse;        // kDz
  const float* loss;       // kDz, K = 0
  const float* d_loss;
  const float* d_lse;
  int direct[2];           // kGrad, dx and dW: stored as bf16; otherwise fp32 partials
  int accumulate;          // dx partials are added to those of the piece before
  const float* dx_part;    // [splits, T, D]
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

MOE_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 8 columns of a warp's TMEM lanes, as tmem_ld_32cols.
MOE_DEV void tmem_ld_8cols(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

MOE_DEV long long load_index(const void* p, int is64, size_t i) {
  return is64 ? static_cast<const long long*>(p)[i] : static_cast<const int*>(p)[i];
}

// Order of a target among those of its row: first those of the columns that one
// half of the epilogue has (bit 7 of the id), then the other's, each by column.
// No target: all ones.
__host__ MOE_DEV uint32_t target_key(uint32_t id, uint32_t entry) { return (id >> 7 & 1u) << 30 | id << 8 | entry; }

// A row's targets in one half of the columns, in ascending order, four at a time:
// most runs of the vocabulary have fewer of a row.  (A key asked for at every step,
// three ahead, made the next step wait for it: 315 us instead of 288, 32768 x 768 x
// 8192 with 64 a token; both halves' keys in one list, one ahead: 1790 us instead of
// 1490, 32768 x 768 x 50001.)
struct Targets {
  uint32_t now, next1, next2, next3;  // id << 8 | entry, or more than any of those
  int left, pos;                      // of these four; the key after them

  MOE_DEV int id() const { return static_cast<int>(now >> 8); }
  MOE_DEV int entry() const { return static_cast<int>(now & 255u); }
  MOE_DEV void load(const VocabArgs& p, int row, int half) {
    const uint32_t* k = p.keys + static_cast<size_t>(row) * p.K;
    auto key = [&](int i) { return i < p.K ? k[i] - (static_cast<uint32_t>(half) << 30) : 0xffffffffu; };
    now = key(pos);
    next1 = key(pos + 1);
    next2 = key(pos + 2);
    next3 = key(pos + 3);
    pos += 4;
    left = 4;
  }
  MOE_DEV void step(const VocabArgs& p, int row, int half) {
    now = next1;
    next1 = next2;
    next2 = next3;
    next3 = 0xffffffffu;
    if (--left == 0 && pos < p.K) load(p, row, half);
  }
  // From the first target at or past column `col`.
  MOE_DEV void start(const VocabArgs& p, int row, int half, int col) {
    now = next1 = next2 = next3 = 0xffffffffu;
    left = 4;
    pos = p.K;
    if (row >= p.T) return;
    if (p.K == 0) {
      const long long l = load_index(p.labels, p.labels64, row);
      if (l >= col && l < p.V && (l >> 7 & 1) == half) now = static_cast<uint32_t>(l) << 8;
      return;
    }
    if (p.keys == nullptr) return;  // kDz: those come after it
    const uint32_t* k = p.keys + static_cast<size_t>(row) * p.K;
    const uint32_t want = static_cast<uint32_t>(half) << 30 | static_cast<uint32_t>(col) << 8;
    // eight probes at once: two or three rounds of L2's latency, not six to eight
    int lo = 0, hi = p.K;  // the answer lies in [lo, hi]
    while (lo < hi) {
      const int by = (hi - lo + 8) / 9;
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k[min(lo + by * (i + 1), hi) - 1];
      int less = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) less += lo + by * (i + 1) <= hi && v[i] < want ? 1 : 0;
      if (less < 8) hi = min(hi, lo + by * (less + 1) - 1);
      lo += by * less;
    }
    pos = lo;
    if (pos < p.K) load(p, row, half);
  }
};

// a of a row: of cross entropy d_loss + d_lse, where a token without a loss has no
// d_loss.
MOE_DEV float factor_of(const VocabArgs& p, int row) {
  if (p.K > 0) return p.row_a[row];
  const long long id = load_index(p.labels, p.labels64, row);
  return (id >= 0 && id < p.V ? p.d_loss[row] : 0.f) + (p.d_lse ? p.d_lse[row] : 0.f);
}

// dz at a token's label, d_loss (q - 1) + d_lse q with q - 1 = expm1(-loss), as
// bf16.  (No gradient: 0 whatever the loss is, infinite or no number.)
MOE_DEV uint16_t at_label(const VocabArgs& p, int row) {
  const float d = p.d_loss[row], e = p.d_lse ? p.d_lse[row] : 0.f, loss = p.loss[row];
  const float v = (d == 0.f ? 0.f : d * expm1f(-loss)) + (e == 0.f ? 0.f : e * expf(-loss));
  return static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xffffu);
}

// Element j of 32 registers, by halves.  (Through the warp's buffer in shared
// memory, which the MMAs read at the same time: 400 us instead of 340, 32768 x 768
// x 8192 with 64 targets a token; without targets 262.)
MOE_DEV uint32_t pick(const uint32_t (&v)[32], int j) {
  uint32_t t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) t[i] = j & 16 ? v[i + 16] : v[i];
#pragma unroll
  for (int h = 8; h > 0; h >>= 1)
#pragma unroll
    for (int i = 0; i < h; ++i) t[i] = j & h ? t[i + h] : t[i];
  return t[0];
}

// 128 bytes into a lane's row of its warp's buffer.
MOE_DEV void put_row(uint8_t* mine, const uint32_t (&w)[32]) {
  const uint32_t turn = lane_id() & 7u;
#pragma unroll
  for (uint32_t c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(mine + ((c ^ turn) << 4)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

// kParts: a logit is the sum of p.parts sums over D.
template <int kMode, bool kParts>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_kernel(const __grid_constant__ CUtensorMap mapX, const __grid_constant__ CUtensorMap mapW,
                 const __grid_constant__ CUtensorMap mapZ, const __grid_constant__ CUtensorMap mapOut0,
                 const __grid_constant__ CUtensorMap mapOut1, const VocabArgs p) {
  extern __shared__ uint8_t vocab_smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(vocab_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t smem_base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int pair = static_cast<int>(cluster_id_x());
  const int npairs = static_cast<int>(num_clusters_x());

  if (warp == 0 && lane == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(smem_u32(&ctl.full[st]), 1);
      mbar_init(smem_u32(&ctl.empty[st]), 1);
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
  griddep_wait();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem_base = ctl.tmem_base;
  volatile int* abort_flag = &ctl.abort;
  unsigned int* dev_err = p.dev_err;
  Walk<kMode> walk;
  Unit u;

  if (warp == 0) {
    // ===================== TMA producer (both CTAs) =====================
    if (lane == 0) {
      // What is loaded is read again by other pairs, what is stored is for later.
      // Kept over it, kDz takes 1486 us instead of 1493 (32768 x 768 x 50001) and
      // 2328 instead of 2392 (8192 x 2048 x 131072), kStats 1242 and 2133 instead of
      // 1266 and 2161, kGrad 2627 and 4586 instead of 2691 and 4808.
      const uint64_t pol = l2_policy_evict_last();
      auto load_tokens = [&](uint32_t dst, const CUtensorMap& map, int row, int block, uint32_t full) {
        tma_load_3d_pair(dst, &map, full, 0, row, block, pol);
        if (p.box < 128) tma_load_3d_pair(dst + kOperandBytes / 2, &map, full, 0, row, block + 1, pol);
      };
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
      while (ok && walk.next(p, pair, npairs, u)) {
        const bool dw = kMode == kGrad && u.which == 1;
        const int m0 = u.m * kTile + 128 * rank, n0 = u.n * kTile + 128 * rank;
        // rows past the last token are not loaded, nor zeroed: they hold anything, and
        // nothing reads what comes of them
        const bool here = dw || m0 < p.T, peer = dw || u.m * kTile + 128 < p.T;
        const uint32_t bytes = 256 * ((peer ? 2 : 1) * p.box + 2 * (dw ? p.box : 128));
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          if (!mbar_wait_cluster(smem_u32(&ctl.empty[stage]), phase ^ 1u, abort_flag, dev_err)) {
            ok = false;
            break;
          }
          const uint32_t full_leader = map_to_cta(smem_u32(&ctl.full[stage]), 0);
          const uint32_t sa = smem_base + stage * kStageBytes, sb = sa + kOperandBytes;
          if (leader) mbar_arrive_expect_tx(smem_u32(&ctl.full[stage]), bytes);
          if constexpr (kMode == kGrad) {
            if (u.which == 0) {  // dz rows, W's rows as k
              if (here) load_tokens(sa, mapZ, m0, kb * (kBK / 64), full_leader);
              tma_load_3d_pair(sb, &mapW, full_leader, 0, p.v0 + kb * kBK, n0 / 64, pol);
            } else {  // dz columns, tokens as k
              load_tokens(sa, mapZ, kb * kBK, m0 / 64, full_leader);
              load_tokens(sb, mapX, kb * kBK, n0 / 64, full_leader);
            }
          } else {
            if (here) load_tokens(sa, mapX, m0, kb * (kBK / 64), full_leader);
            tma_load_3d_pair(sb, &mapW, full_leader, 0, p.v0 + n0, kb * (kBK / 64), pol);
          }
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) {
        // Let the copies already in flight land before the CTA exits.
        int st = stage;
        uint32_t ph = phase;
        for (int i = 0; i < kStages && i < issued; ++i) {
          if (--st < 0) {
            st = kStages - 1;
            ph ^= 1u;
          }
          volatile int local_abort = 0;
          mbar_wait_cluster(smem_u32(&ctl.full[st]), ph, &local_abort, dev_err);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ===================== MMA issuer (leader only) =====================
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0;
      int i = 0;
      bool ok = true;
      const int parts = kParts ? p.parts : 1;
      for (int part = parts; ok; ++i) {
        if (part == parts) {
          if (!walk.next(p, pair, npairs, u)) break;
          part = 0;
        }
        const int buf = i & 1;
        if (!mbar_wait_cluster(smem_u32(&ctl.tempty[buf]), ((i >> 1) & 1) ^ 1u, abort_flag, dev_err)) break;
        tc_fence_after_sync();
        const int first = kParts ? u.kb1 * part / parts : u.kb0;
        const int end = kParts ? u.kb1 * (part + 1) / parts : u.kb1;
        ++part;
        const uint32_t d_tmem = tmem_base + buf * 256;
        // kGrad: B is N-major, A M-major where the tokens are the reduction
        const uint32_t a_mn = kMode == kGrad && u.which == 1, b_mn = kMode == kGrad;
        const uint32_t idesc = idesc_bf16_f32_ab(kTile, kTile, a_mn, b_mn);
        const uint32_t a_lbo = a_mn ? 16384 : 16;
        for (int kb = first; kb < end; ++kb) {
          if (!mbar_wait_cluster(smem_u32(&ctl.full[stage]), phase, abort_flag, dev_err)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sa = smem_base + stage * kStageBytes, sb = sa + kOperandBytes;
          const int slices = kMode == kGrad && u.which == 1 ? p.box / 16 : kBK / 16;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            if (kk >= slices) break;
            const uint32_t k_major = (kk >> 2) * 16384 + (kk & 3) * 32, mn_major = kk * 2048;
            const uint64_t adesc = smem_desc_sw128(sa + (a_mn ? mn_major : k_major), a_lbo, 1024);
            const uint64_t bdesc = smem_desc_sw128(sb + (b_mn ? mn_major : k_major), b_mn ? 16384 : 16, 1024);
            umma_bf16_pair(d_tmem, adesc, bdesc, idesc, (kb != first || kk != 0) ? 1u : 0u);
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
  } else {
    // ===================== epilogue (both CTAs) =====================
    // Warp w owns TMEM lanes 32 (w % 4) .. + 31, a row a lane, and half
    // (w - 2) / 4 of the tile's columns.  It reads its 128 columns in one burst
    // and hands the accumulator back before any math.
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int c_first = half * 128;
    const uint32_t tempty_leader0 = map_to_cta(smem_u32(&ctl.tempty[0]), 0);
    const uint32_t tempty_leader1 = map_to_cta(smem_u32(&ctl.tempty[1]), 0);
    uint8_t* box = smem + kStages * kStageBytes + (warp - 2) * kBoxBytes;
    uint8_t* mine = box + lane * 128;  // a lane's row of it
    float run_max = -INFINITY, run_sum = 0.f;
    Targets tg;
    float row_a = 0.f, row_l = 0.f;
    int i = 0;  // sums taken out of TMEM
    while (walk.next(p, pair, npairs, u)) {
      const int warp_row0 = u.m * kTile + 128 * rank + q * 32;
      const int row = warp_row0 + lane;
      const int col0 = u.n * kTile + c_first;  // first column of this warp (of the piece, in kDz)
      if constexpr (kMode != kGrad) {
        if (u.first) {
          tg.start(p, row, half, p.v0 + col0);
          run_max = -INFINITY;
          run_sum = 0.f;
          if constexpr (kMode == kDz) {
            row_a = row < p.T ? factor_of(p, row) : 0.f;
            row_l = row < p.T ? p.lse[row] * kLog2e : 0.f;
          }
        }
      }
      uint32_t acc[kBoxes][32];
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + c_first;
      auto filled = [&] {
        const bool got = mbar_wait_cluster(smem_u32(&ctl.tfull[i & 1]), (i >> 1) & 1, abort_flag, dev_err);
        const bool all = __all_sync(0xffffffffu, got);
        tc_fence_after_sync();
        return all;
      };
      auto hand_back = [&] {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(i & 1 ? tempty_leader1 : tempty_leader0);
        ++i;
      };
      bool ok = filled();
      if (!ok) break;
#pragma unroll
      for (int b = 0; b < kBoxes; ++b) tmem_ld_32cols(taddr + (i & 1) * 256 + b * 32, acc[b]);
      tmem_ld_wait();
      hand_back();
      if constexpr (kParts) {
        // (8 columns at a time: 16 do not fit beside the 128 in registers)
#pragma unroll 1
        for (int part = 1; part < p.parts; ++part) {
          if (!(ok = filled())) break;
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            uint32_t more[8];
            tmem_ld_8cols(taddr + (i & 1) * 256 + g * 8, more);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t& to = acc[g / 4][g % 4 * 8 + j];
              to = __float_as_uint(__uint_as_float(to) + __uint_as_float(more[j]));
            }
          }
          hand_back();
        }
        if (!ok) break;
      }

      if constexpr (kMode == kStats) {
        if (col0 + 128 > p.V) {  // columns past the vocabulary
#pragma unroll
          for (int b = 0; b < kBoxes; ++b)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (col0 + b * 32 + j >= p.V) acc[b][j] = 0xff800000u;
        }
#pragma unroll
        for (int b = 0; b < kBoxes; ++b) {
          // each turn takes at most one target of a lane out of the box
          const int begin = col0 + b * 32;
          while (__any_sync(0xffffffffu, tg.id() < begin + 32)) {
            const float z = __uint_as_float(pick(acc[b], tg.id() - begin));
            if (tg.id() < begin + 32) {
              p.target[p.K == 0 ? static_cast<size_t>(row) : static_cast<size_t>(row) * p.K + tg.entry()] = z;
              tg.step(p, row, half);
            }
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int b = 0; b < kBoxes; ++b)
#pragma unroll
          for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(acc[b][j]));
        const float tile_max = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c;
        const float new_max = fmaxf(run_max, tile_max);
        const float ref = new_max == -INFINITY ? 0.f : new_max;  // nothing but -inf so far
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < kBoxes; ++b)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[j & 3] += exp2_fast(fmaf(__uint_as_float(acc[b][j]), p.c, -ref));
        run_sum = run_sum * exp2_fast(run_max - ref) + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
        run_max = new_max;
        if (u.last && row < p.T)
          p.part[static_cast<size_t>(2 * u.slot + half) * p.rows_padded + row] = make_float2(run_max, run_sum);
      } else if constexpr (kMode == kDz) {
        if (warp_row0 >= p.T) continue;
#pragma unroll
        for (int b = 0; b < kBoxes; b += 2) {
          const int cc = col0 + b * 32;
          if (cc >= p.Vcp) break;
          uint32_t packed[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float lo = row_a * exp2_fast(fmaf(__uint_as_float(acc[b + j / 16][2 * (j & 15)]), p.c, -row_l));
            const float hi = row_a * exp2_fast(fmaf(__uint_as_float(acc[b + j / 16][2 * (j & 15) + 1]), p.c, -row_l));
            packed[j] = row_a == 0.f ? 0u : pack_bf16x2(lo, hi);  // whatever a row without a loss holds
          }
          if (cc + 64 > p.Vc) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (cc + 2 * j >= p.Vc) packed[j] = 0u;
              else if (cc + 2 * j + 1 >= p.Vc) packed[j] &= 0xffffu;
            }
          }
          bulk_wait_group_read0();
          __syncwarp();
          put_row(mine, packed);
          const int end = p.v0 + cc + 64;
          if (tg.id() < end) {
            const int j = tg.id() - (end - 64);
            *reinterpret_cast<uint16_t*>(mine + (((j >> 3) ^ (lane & 7)) << 4) + (j & 7) * 2) = at_label(p, row);
            tg.step(p, row, half);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&mapOut0, smem_u32(box), 0, warp_row0, cc / 64);
            bulk_commit_group();
          }
        }
      } else {
        const int rows = u.which == 0 ? p.T : p.Vc;
        if (warp_row0 >= rows) continue;
        const int out_row = u.which == 0 ? warp_row0 : p.v0 + warp_row0;
        const CUtensorMap* map = u.which == 0 ? &mapOut0 : &mapOut1;
        if (p.direct[u.which]) {
#pragma unroll
          for (int b = 0; b < kBoxes; b += 2) {
            const int cc = col0 + b * 32;
            if (cc >= p.D) break;
            uint32_t packed[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
              packed[j] = pack_bf16x2(__uint_as_float(acc[b + j / 16][2 * (j & 15)]),
                                      __uint_as_float(acc[b + j / 16][2 * (j & 15) + 1]));
            bulk_wait_group_read0();
            __syncwarp();
            put_row(mine, packed);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(map, smem_u32(box), cc, out_row);
              bulk_commit_group();
            }
          }
          continue;
        }
#pragma unroll
        for (int b = 0; b < kBoxes; ++b) {
          const int cc = col0 + b * 32;
          if (cc >= p.D) break;
          if (u.which == 0 && p.accumulate && row < p.T) {
            const float4* before = reinterpret_cast<const float4*>(
                p.dx_part + (static_cast<size_t>(u.split) * p.T + row) * p.D + cc);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const float4 f = before[v];
              acc[b][4 * v] = __float_as_uint(__uint_as_float(acc[b][4 * v]) + f.x);
              acc[b][4 * v + 1] = __float_as_uint(__uint_as_float(acc[b][4 * v + 1]) + f.y);
              acc[b][4 * v + 2] = __float_as_uint(__uint_as_float(acc[b][4 * v + 2]) + f.z);
              acc[b][4 * v + 3] = __float_as_uint(__uint_as_float(acc[b][4 * v + 3]) + f.w);
            }
          }
          bulk_wait_group_read0();
          __syncwarp();
          put_row(mine, acc[b]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(map, smem_u32(box), cc, out_row, u.split);
            bulk_commit_group();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group0();
    __syncwarp();
  }

  // Both CTAs done with TMEM and with each other's barriers before freeing.
  tc_fence_before_sync();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Rows: what the products need of them and what is left to do after them
// ---------------------------------------------------------------------------
constexpr int kRowWarps = 8;

// (maximum, sum) pairs joined; an empty one is (-inf, 0).
MOE_DEV void join(float& m, float& s, float m2, float s2) {
  const float n = fmaxf(m, m2);
  const float ref = n == -INFINITY ? 0.f : n;
  s = s * exp2_fast(m - ref) + s2 * exp2_fast(m2 - ref);
  m = n;
}

// The teacher's entries of one row, by one warp: entry j = lane + 32 i in slot i
// of kSlots = ceil(K / 32), rounded up to a power of two.  Entries outside the
// vocabulary or of -inf are none.
template <int kSlots>
struct Teacher {
  float p[kSlots];      // probability (0 where there is none)
  float log_p[kSlots];
  int id[kSlots];       // or -1
};

MOE_DEV float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
MOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

MOE_DEV float teacher_logit(const VocabTargets& t, size_t at) {
  return t.logits_fp32 ? static_cast<const float*>(t.logits)[at]
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(t.logits)[at]);
}

template <int kSlots>
MOE_DEV void read_teacher(const VocabTargets& t, int row, int V, float inv_tau, Teacher<kSlots>& out) {
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    out.id[i] = -1;
    out.p[i] = -INFINITY;
    const int j = lane + 32 * i;
    if (j < t.K) {
      const size_t at = static_cast<size_t>(row) * t.K + j;
      const long long id = load_index(t.ids, t.ids64, at);
      const float l = teacher_logit(t, at);
      if (id >= 0 && id < V) {
        out.id[i] = static_cast<int>(id);
        out.p[i] = l;
      }
    }
    top = fmaxf(top, out.p[i]);
  }
  top = warp_max(top);
  const float ref = top == -INFINITY ? 0.f : top;
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    // (the difference first, and of halves: neither it nor a logit over the
    // temperature need lie in fp32's range)
    out.log_p[i] = (0.5f * out.p[i] - 0.5f * ref) * (2.f * inv_tau);
    out.p[i] = expf(out.log_p[i]);
    total += out.p[i];
  }
  total = warp_sum(total);
  const float log_total = logf(total), inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    out.p[i] *= inv;
    out.log_p[i] -= log_total;
  }
}

// Sorts 32 kSlots keys, key lane + 32 i in k[i], by a bitonic network: distances
// from 32 on between a lane's own registers, shorter ones between lanes.
template <int kSlots>
MOE_DEV void sort_keys(uint32_t (&k)[kSlots]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32 * kSlots; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (d >= 32) {
          const int o = i ^ (d >> 5);
          if (o < i) continue;
          const bool up = ((32 * i) & size) == 0;
          const uint32_t lo = min(k[i], k[o]), hi = max(k[i], k[o]);
          k[i] = up ? lo : hi;
          k[o] = up ? hi : lo;
        } else {
          const uint32_t other = __shfl_xor_sync(0xffffffffu, k[i], d);
          const bool up = ((32 * i + lane) & size) == 0, first = (lane & d) == 0;
          k[i] = first == up ? min(k[i], other) : max(k[i], other);
        }
      }
}

// Forward of distillation: the rows' sorted keys.
template <int kSlots>
__global__ void __launch_bounds__(32 * kRowWarps) vocab_keys_kernel(VocabTargets t, int T, int V, uint32_t* keys,
                                                                    float* target) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, row = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (row >= T) return;
  uint32_t k[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int j = lane + 32 * i;
    const size_t at = static_cast<size_t>(row) * t.K + j;
    const long long id = j < t.K ? load_index(t.ids, t.ids64, at) : -1;
    const bool known = id >= 0 && id < V;
    k[i] = known ? target_key(static_cast<uint32_t>(id), static_cast<uint32_t>(j)) : 0xffffffffu;
    if (j < t.K && !known) target[at] = 0.f;
  }
  sort_keys(k);
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (lane + 32 * i < t.K) keys[static_cast<size_t>(row) * t.K + lane + 32 * i] = k[i];
}

// Every kWarps-th of a row's pairs from i on, kBatch of them in flight.
template <int kBatch, int kWarps>
MOE_DEV void join_pairs(const float2* row, int i, int parts, int rows_padded, float& m, float& s) {
  float2 v[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) v[j] = row[static_cast<size_t>(min(i + j * kWarps, parts - 1)) * rows_padded];
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    if (i + j * kWarps < parts) join(m, s, v[j].x, v[j].y);
}

// Joins a row's (maximum, sum) pairs and writes lse and the loss: 32 rows a
// block, the pairs dealt to its warps, then the rows.  With the sum s relative
// to 2^m,
//   lse - z / temperature = ln 2 (log2 s - (c z - m)),
// where c z - m is one fused product: for a target that outweighs the rest both
// terms are next to 0, and the difference of the rounded lse and z, which would
// be off by 2^-24 of their size, is never formed.
// kWarps: 32 below 4096 rows, where few blocks have many pairs (a call of 219 x 576 x
// 143711: 43.5 us, with 16 warps 45.1), 8 from 12288 rows on, where more warps only wait
// for one another (32768 x 64 x 512 with 64 entries: 82, with 16 84, with 32 91), 16
// between (7048 x 192 x 449 with 141 entries: 46, with 8 54, with 32 48).
template <int kSlots, int kWarps>
__global__ void __launch_bounds__(32 * kWarps)
    vocab_finish_kernel(const float2* part, int parts, int rows_padded, VocabTargets t, const float* target, int T, int V,
                        float c, float inv_tau, float* loss, float* lse) {
  __shared__ float2 got[kWarps][33];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * 32;
  // lane: a row of the block; warp: every kWarps-th pair of it
  float m = -INFINITY, s = 0.f;
  if (row0 + lane < T) {
    const float2* mine = part + row0 + lane;
    int i = warp;
    for (; i + 12 * kWarps < parts; i += 16 * kWarps) join_pairs<16, kWarps>(mine, i, parts, rows_padded, m, s);
    for (; i < parts; i += 4 * kWarps) join_pairs<4, kWarps>(mine, i, parts, rows_padded, m, s);
  }
  got[warp][lane] = make_float2(m, s);
  __syncthreads();
  if constexpr (kSlots == 0 && kWarps <= 16) {
    // a lane a row, in the order of the shuffles below, so that a teacher of one
    // entry gets a label's bits
    const int row = row0 + lane;
    if (warp > 0 || row >= T) return;
    float2 v[kWarps];
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v[i] = got[i][lane];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < o; ++i) join(v[i].x, v[i].y, v[i + o].x, v[i + o].y);
    m = v[0].x;
    const float log_s = log2f(v[0].y);
    const long long id = load_index(t.ids, t.ids64, row);
    lse[row] = (m + log_s) * kLn2;
    loss[row] = id >= 0 && id < V ? (log_s - fmaf(target[row], c, -m)) * kLn2 : 0.f;
  } else {
    // a warp a row
    for (int r = warp; r < 32; r += kWarps) {
      const int row = row0 + r;
      if (row >= T) return;
      m = lane < kWarps ? got[lane % kWarps][r].x : -INFINITY;
      s = lane < kWarps ? got[lane % kWarps][r].y : 0.f;
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        join(m, s, m2, s2);
      }
      m = __shfl_sync(0xffffffffu, m, 0);
      s = __shfl_sync(0xffffffffu, s, 0);
      const float log_s = log2f(s);
      if (lane == 0) lse[row] = (m + log_s) * kLn2;
      if constexpr (kSlots == 0) {
        if (lane == 0) {
          const long long id = load_index(t.ids, t.ids64, row);
          loss[row] = id >= 0 && id < V ? (log_s - fmaf(target[row], c, -m)) * kLn2 : 0.f;
        }
      } else {
        Teacher<kSlots> te;
        read_teacher(t, row, V, inv_tau, te);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          const int j = lane + 32 * i;
          if (j < t.K && te.id[i] >= 0 && te.p[i] != 0.f)
            sum += te.p[i] * (te.log_p[i] + (log_s - fmaf(target[static_cast<size_t>(row) * t.K + j], c, -m)) * kLn2);
        }
        sum = warp_sum(sum);
        if (lane == 0) loss[row] = sum;
      }
    }
  }
}

// Backward of distillation: a of each row; a token without entries has none.
__global__ void __launch_bounds__(32 * kRowWarps)
    vocab_distill_rows_kernel(const float* d_loss, VocabTargets t, int T, int V, float inv_tau, float* row_a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, row = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (row >= T) return;
  bool any = false;
  for (int j0 = 0; j0 < t.K && !any; j0 += 32) {
    const int j = min(j0 + lane, t.K - 1);
    const size_t at = static_cast<size_t>(row) * t.K + j;
    const long long id = load_index(t.ids, t.ids64, at);
    any = __any_sync(0xffffffffu, id >= 0 && id < V && teacher_logit(t, at) != -INFINITY);
  }
  if (lane == 0) row_a[row] = any ? d_loss[row] * inv_tau : 0.f;
}

// dz at the teacher's entries of a piece's columns,
//   d_loss / temperature (q - p),
// p summed over the entries of one id, in place of what the product's epilogue
// has stored there.  (In the epilogue itself, a row's entries one after the
// other, 64 of them cost 40 us of 425 at 8192 x 768 x 50001, and 225 of them 34 of
// 72 at 353 x 320 x 78226.)  No programmatic launch: blocks that start while the
// product still holds most SMs crowd the few that are free, and 353 rows of 225
// entries then take 68 us instead of 22.
template <int kSlots>
__global__ void __launch_bounds__(32 * kRowWarps)
    vocab_distill_targets_kernel(const float* row_a, const float* lse, const float* target, VocabTargets t, int T, int V,
                                 float inv_tau, int v0, int Vc, uint16_t* dz) {
  __shared__ uint32_t ids[kRowWarps][32 * kSlots];
  __shared__ float prob[kRowWarps][32 * kSlots];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * kRowWarps + warp;
  if (row >= T) return;
  const float d = row_a[row], l = lse[row];
  if (d == 0.f) return;
  Teacher<kSlots> te;
  read_teacher(t, row, V, inv_tau, te);
  uint32_t k[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    prob[warp][lane + 32 * i] = te.p[i];
    k[i] = te.id[i] < 0 ? 0xffffffffu : static_cast<uint32_t>(te.id[i]) << 8 | static_cast<uint32_t>(lane + 32 * i);
  }
  sort_keys(k);
  __syncwarp();
  // entries of one id lie side by side: the first of them writes for all
  bool again = false;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    ids[warp][lane + 32 * i] = k[i];
    const uint32_t left = __shfl_up_sync(0xffffffffu, k[i], 1), last = __shfl_sync(0xffffffffu, k[i > 0 ? i - 1 : 0], 31);
    const uint32_t before = lane > 0 ? left : i > 0 ? last : 0xffffffffu;
    again |= k[i] != 0xffffffffu && before >> 8 == k[i] >> 8;
  }
  again = __any_sync(0xffffffffu, again);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const uint32_t id = k[i] >> 8;
    const int at = lane + 32 * i, column = static_cast<int>(id) - v0;
    if (k[i] == 0xffffffffu || column < 0 || column >= Vc) continue;
    float p = prob[warp][k[i] & 255u];
    if (again) {
      if (at > 0 && ids[warp][at - 1] >> 8 == id) continue;
      for (int a = at + 1; a < 32 * kSlots && ids[warp][a] >> 8 == id; ++a) p += prob[warp][ids[warp][a] & 255u];
    }
    const float q = expf(target[static_cast<size_t>(row) * t.K + (k[i] & 255u)] * inv_tau - l);
    dz[(static_cast<size_t>(column >> 6) * T + row) * 64 + (column & 63)] =
        static_cast<uint16_t>(pack_bf16x2(d * (q - p), 0.f) & 0xffffu);
  }
}

// bf16 sums of fp32 partials [n_parts, n] in their order, n a multiple of 8: of dx,
// then of dW, by `blocks` blocks each.
struct Sum {
  const float* part;
  int n_parts, blocks;
  size_t n;
  uint16_t* out;
};

__global__ void __launch_bounds__(256) vocab_sum_kernel(Sum x, Sum w) {
  griddep_launch_dependents();
  griddep_wait();
  const bool of_x = static_cast<int>(blockIdx.x) < x.blocks;
  const Sum& q = of_x ? x : w;
  const size_t i = (static_cast<size_t>(of_x ? blockIdx.x : blockIdx.x - x.blocks) * 256 + threadIdx.x) * 8;
  if (i >= q.n) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 4
  for (int s = 0; s < q.n_parts; ++s) {
    const float4* f = reinterpret_cast<const float4*>(q.part + static_cast<size_t>(s) * q.n + i);
    const float4 u = f[0], v = f[1];
    a.x += u.x, a.y += u.y, a.z += u.z, a.w += u.w;
    b.x += v.x, b.y += v.y, b.z += v.z, b.w += v.w;
  }
  *reinterpret_cast<uint4*>(q.out + i) =
      make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
std::mutex g_mu;
struct Setup {
  int pairs[3] = {0, 0, 0};  // co-resident CTA pairs of each mode, with parts or without
  unsigned int* dev_err = nullptr;
};
Setup g_setup[64];

const void* kernel_of(int mode, bool parts) {
  return mode == kStats ? parts ? reinterpret_cast<const void*>(vocab_kernel<kStats, true>)
                                : reinterpret_cast<const void*>(vocab_kernel<kStats, false>)
         : mode == kDz  ? parts ? reinterpret_cast<const void*>(vocab_kernel<kDz, true>)
                                : reinterpret_cast<const void*>(vocab_kernel<kDz, false>)
                        : reinterpret_cast<const void*>(vocab_kernel<kGrad, false>);
}

cudaLaunchConfig_t pair_config(int pairs, cudaStream_t s, cudaLaunchAttribute (&attr)[2], bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cfg;
}

cudaError_t setup(Setup* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mu);
  Setup& st = g_setup[dev];
  if (st.pairs[kGrad] == 0) {
    Setup got;
    const int sms = current_device_sms();
    if (sms < 2) return cudaErrorInvalidDevice;
    if ((e = device_error_address(&got.dev_err)) != cudaSuccess) return e;
    for (int i = 0; i < 6; ++i) {
      const int mode = i / 2;
      const void* kernel = kernel_of(mode, i % 2 != 0);
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      if (e != cudaSuccess) return e;
      cudaLaunchAttribute attr[2];
      cudaLaunchConfig_t cfg = pair_config(sms / 2, nullptr, attr, false);
      int fit = 0;
      e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (fit < 1) return cudaErrorInvalidConfiguration;
      got.pairs[mode] = i % 2 ? std::min(got.pairs[mode], fit) : fit;
    }
    st = got;
  }
  *out = st;
  return cudaSuccess;
}

template <int kMode>
cudaError_t launch_vocab(int pairs, const CUtensorMap& x, const CUtensorMap& w, const CUtensorMap& z,
                         const CUtensorMap& out0, const CUtensorMap& out1, const VocabArgs& a, cudaStream_t s, bool pdl) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pair_config(pairs, s, attr, pdl);
  auto* k = vocab_kernel<kMode, false>;
  if constexpr (kMode != kGrad)
    if (a.parts > 1) k = vocab_kernel<kMode, true>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, x, w, z, out0, out1, a);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t padded(size_t n) { return (n + 255) / 256 * 256; }

// Takes regions of the workspace one after the other.
struct Take {
  uint8_t* base;
  size_t off = 0;
  template <typename Tp>
  Tp* get(size_t n) {
    Tp* p = reinterpret_cast<Tp*>(base + off);
    off += padded(n * sizeof(Tp));
    return p;
  }
};

struct BackwardRegions {
  float* row_a;
  uint16_t* dz;
  float* dx_part;
  float* dw_part;
};
size_t backward_regions(uint8_t* base, int T, int D, int V, int K, const BackwardPlan& b, BackwardRegions* r) {
  Take t{base};
  const size_t rows = static_cast<size_t>(T);
  r->row_a = t.get<float>(K == 0 ? 0 : rows);
  r->dz = t.get<uint16_t>(rows * b.piece);
  r->dx_part = t.get<float>(b.pieces > 1 || b.splits_x > 1 ? rows * D * b.splits_x : 0);
  r->dw_part = t.get<float>(b.splits_w > 1 ? static_cast<size_t>(V) * D * b.splits_w : 0);
  return t.off;
}

// Sums that a logit is made of.  The tensor cores add 16 products at a time to the
// sum so far and cut the result to 24 bits, towards zero, where fp32 arithmetic
// rounds it: a sum of n products of random sign comes out about 1e-9 n of itself too
// small, of products of one sign two to four times that (3.2e-5 at 8192).  So at most
// kPartBlocks k blocks, 896 products, are summed there, and the parts are added in
// fp32: a logit is off by less than 1e-6 of the size of its sums (one sign: 2e-6 of
// itself) at any width.
// (8192 x 1024 x 50001 in two parts: 490 us, in one 460; 8192 x 4096 x 30001 in five
// 1145, in one 1125; 4096 x 4096 x 30001 backward 1787 and 1770.  Parts of at most 512
// products have half the error, but take 1490 us instead of 1390 for 32768 x 768 x
// 50001; parts of 1024 save nothing but at 1024, and there a logit is 1e-6 off.)
constexpr int kPartBlocks = 7;
int parts_of(int D) { return ceil_div(ceil_div(D, kBK), kPartBlocks); }

// Rows of a box of tokens: 128, with two blocks of columns, or as many as there
// are (in slices of 16 of a reduction over them), with one.  TMA fills what lies
// outside a tensor with zeros, which takes longer than loading as much (forward of
// 8 x 704 x 194036: 78 us with 120 rows of zeros in every box, 58 so; two boxes of
// one block instead of one of two throughout: 1480 us at 32768 x 768 x 50001 instead
// of 1360).
int token_box(int T) { return T < 128 ? (T + 15) / 16 * 16 : 128; }
int box_blocks(int box) { return box < 128 ? 1 : 2; }

// The kernel for a teacher of K entries.
template <typename Kernel>
Kernel by_slots(int K, Kernel k1, Kernel k2, Kernel k4, Kernel k8) {
  return K <= 32 ? k1 : K <= 64 ? k2 : K <= 128 ? k4 : k8;
}

template <int kWarps>
cudaError_t launch_finish(const VocabForward& a, const VocabArgs& v, const ForwardPlan& f, float inv_tau, cudaStream_t s) {
  auto* k = v.K == 0 ? vocab_finish_kernel<0, kWarps>
                     : by_slots(v.K, vocab_finish_kernel<1, kWarps>, vocab_finish_kernel<2, kWarps>,
                                vocab_finish_kernel<4, kWarps>, vocab_finish_kernel<8, kWarps>);
  return launch_kernel(k, dim3(ceil_div(a.T, 32)), dim3(32 * kWarps), 0, s, true, static_cast<const float2*>(v.part),
                       2 * f.runs, f.rows_padded, a.targets, static_cast<const float*>(v.target), a.T, a.V, v.c, inv_tau,
                       a.loss, a.lse);
}

Sum sum_of(const float* part, int n_parts, size_t n, uint16_t* out) {
  return Sum{part, n_parts, ceil_div(static_cast<long>(n / 8), 256), n, out};
}

}  // namespace

size_t vocab_forward_workspace_bytes(int T, int D, int V, int K) {
  const ForwardPlan f = forward_plan(T, V);
  Take t{nullptr};
  t.get<float2>(static_cast<size_t>(2) * f.runs * f.rows_padded);
  t.get<uint32_t>(static_cast<size_t>(T) * K);
  t.get<float>(K == 0 ? T : 0);
  return t.off;
}

cudaError_t launch_vocab_forward(const VocabForward& a, void* workspace, cudaStream_t s) {
  Setup st;
  cudaError_t e = setup(&st);
  if (e != cudaSuccess) return e;
  const ForwardPlan f = forward_plan(a.T, a.V);
  Take t{static_cast<uint8_t*>(workspace)};
  VocabArgs v = {};
  v.T = a.T;
  v.V = v.Vc = v.Vcp = a.V;
  v.D = a.D;
  v.VocabWork::operator=(forward_work(f, a.D));
  v.c = kLog2e / a.temperature;
  v.parts = parts_of(a.D);
  v.K = a.targets.K;
  v.labels = a.targets.ids;
  v.labels64 = a.targets.ids64;
  v.part = t.get<float2>(static_cast<size_t>(2) * f.runs * f.rows_padded);
  v.rows_padded = f.rows_padded;
  uint32_t* keys = t.get<uint32_t>(static_cast<size_t>(a.T) * v.K);
  v.keys = keys;
  v.target = v.K ? a.target : t.get<float>(a.T);
  v.dev_err = st.dev_err;
  v.box = token_box(a.T);
  CUtensorMap mx, mw;
  if ((e = tensor_map_blocks(&mx, a.x, a.T, a.D, box_blocks(v.box), v.box)) != cudaSuccess) return e;
  if ((e = tensor_map_blocks(&mw, a.W, a.V, a.D, 2, 128)) != cudaSuccess) return e;
  const float inv_tau = 1.f / a.temperature;
  if (v.K) {
    auto* k = by_slots(v.K, vocab_keys_kernel<1>, vocab_keys_kernel<2>, vocab_keys_kernel<4>, vocab_keys_kernel<8>);
    e = launch_kernel(k, dim3(ceil_div(a.T, kRowWarps)), dim3(32 * kRowWarps), 0, s, false, a.targets, a.T, a.V,
                      keys, v.target);
    if (e != cudaSuccess) return e;
  }
  e = launch_vocab<kStats>(std::min(st.pairs[kStats], v.items), mx, mw, mx, mx, mx, v, s, v.K != 0);
  if (e != cudaSuccess) return e;
  return a.T < 4096    ? launch_finish<32>(a, v, f, inv_tau, s)
         : a.T < 12288 ? launch_finish<16>(a, v, f, inv_tau, s)
                       : launch_finish<8>(a, v, f, inv_tau, s);
}

size_t vocab_backward_workspace_bytes(int T, int D, int V, int K) {
  BackwardRegions r;
  return backward_regions(nullptr, T, D, V, K, backward_plan(T, D, V), &r);
}

cudaError_t launch_vocab_backward(const VocabBackward& a, void* workspace, cudaStream_t s) {
  Setup st;
  cudaError_t e = setup(&st);
  if (e != cudaSuccess) return e;
  const int K = a.targets.K;
  const BackwardPlan b = backward_plan(a.T, a.D, a.V);
  BackwardRegions r;
  backward_regions(static_cast<uint8_t*>(workspace), a.T, a.D, a.V, K, b, &r);
  VocabArgs v = {};
  v.T = a.T;
  v.D = a.D;
  v.V = a.V;
  v.c = kLog2e / a.temperature;
  v.parts = parts_of(a.D);
  v.K = K;
  v.labels = a.targets.ids;
  v.labels64 = a.targets.ids64;
  v.row_a = r.row_a;
  v.lse = a.lse;
  v.loss = a.loss;
  v.d_loss = a.d_loss;
  v.d_lse = a.d_lse;
  const bool dx_direct = b.pieces == 1 && b.splits_x == 1, dw_direct = b.splits_w == 1;
  v.direct[0] = dx_direct;
  v.direct[1] = dw_direct;
  v.dx_part = r.dx_part;
  v.dev_err = st.dev_err;
  v.box = token_box(a.T);
  CUtensorMap mx, mw, mz, mz_out, mdx, mdw;
  if ((e = tensor_map_blocks(&mx, a.x, a.T, a.D, box_blocks(v.box), v.box)) != cudaSuccess) return e;
  if ((e = tensor_map_blocks(&mw, a.W, a.V, a.D, 2, 128)) != cudaSuccess) return e;
  e = dx_direct ? tensor_map_2d(&mdx, a.dx, a.T, a.D, 32, 64)
                : tensor_map_f32_3d(&mdx, r.dx_part, a.D, a.T, b.splits_x, 32, 32);
  if (e != cudaSuccess) return e;
  e = dw_direct ? tensor_map_2d(&mdw, a.dW, a.V, a.D, 32, 64)
                : tensor_map_f32_3d(&mdw, r.dw_part, a.D, a.V, b.splits_w, 32, 32);
  if (e != cudaSuccess) return e;
  const float inv_tau = 1.f / a.temperature;
  if (K) {
    e = launch_kernel(vocab_distill_rows_kernel, dim3(ceil_div(a.T, kRowWarps)), dim3(32 * kRowWarps), 0, s, false,
                      a.d_loss, a.targets, a.T, a.V, inv_tau, r.row_a);
    if (e != cudaSuccess) return e;
  }
  for (int i = 0; i < b.pieces; ++i) {
    v.v0 = i * b.piece;
    v.Vc = std::min(b.piece, a.V - v.v0);
    v.Vcp = ceil_div(v.Vc, 64) * 64;
    v.accumulate = i > 0;
    if ((e = tensor_map_block_major(&mz, r.dz, a.T, v.Vcp / 64, v.box, box_blocks(v.box))) != cudaSuccess) return e;
    if ((e = tensor_map_block_major(&mz_out, r.dz, a.T, v.Vcp / 64, 32, 1)) != cudaSuccess) return e;
    v.VocabWork::operator=(dz_work(b, a.D, v.Vc));
    e = launch_vocab<kDz>(std::min(st.pairs[kDz], v.items), mx, mw, mz, mz_out, mz_out, v, s, K != 0 || i > 0);
    if (e != cudaSuccess) return e;
    if (K) {
      auto* k = by_slots(K, vocab_distill_targets_kernel<1>, vocab_distill_targets_kernel<2>,
                         vocab_distill_targets_kernel<4>, vocab_distill_targets_kernel<8>);
      e = launch_kernel(k, dim3(ceil_div(a.T, kRowWarps)), dim3(32 * kRowWarps), 0, s, false,
                        static_cast<const float*>(r.row_a), a.lse, a.target, a.targets, a.T, a.V, inv_tau, v.v0, v.Vc,
                        r.dz);
      if (e != cudaSuccess) return e;
    }
    v.VocabWork::operator=(grad_work(b, a.T, v.Vc));
    e = launch_vocab<kGrad>(std::min(st.pairs[kGrad], v.n_units[0] + v.n_units[1]), mx, mw, mz, mdx, mdw, v, s, true);
    if (e != cudaSuccess) return e;
  }
  if (dx_direct && dw_direct) return cudaSuccess;
  const Sum x = dx_direct ? Sum{} : sum_of(r.dx_part, b.splits_x, static_cast<size_t>(a.T) * a.D, a.dx);
  const Sum w = dw_direct ? Sum{} : sum_of(r.dw_part, b.splits_w, static_cast<size_t>(a.V) * a.D, a.dW);
  return launch_kernel(vocab_sum_kernel, dim3(x.blocks + w.blocks), dim3(256), 0, s, true, x, w);
}

}  // namespace moe
