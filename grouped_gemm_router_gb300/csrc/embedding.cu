// Embedding lookup, out[t] = scale table[ids[t]], and its gradient,
// d_table[v] = (add[v] +) scale sum over {t : ids[t] = v} of d_out[t].
//
// Both are bound by memory.  The lookup gives a row to a few lanes, up to four
// 16-byte pieces each.
//
// The gradient sorts the tokens by id (stable radix sort, up to 9 bits a pass:
// two passes up to 262143 ids).  Then a warp takes four
// sorted tokens and writes the rows of the table whose tokens begin there, sums in
// token order in fp32: no sum depends on timing.  Rows without tokens (zeros, or `add`) are
// most of a large table: all rows are filled with those beside the sort, which
// keeps few SMs busy; the rows with tokens are then written a second time.
// Frequent tokens would leave one warp with thousands of rows to add: aligned
// runs of `chunk` sorted tokens with one id are summed by warps of their own
// beforehand, the long runs are listed, and each is then added by a whole block.
#include <algorithm>
#include <mutex>

#include "moe_device.cuh"
#include "moe_kernels.cuh"

namespace moe {
namespace {

MOE_DEV long long load_id(const void* p, int is64, size_t i) {
  return is64 ? static_cast<const long long*>(p)[i] : static_cast<const int*>(p)[i];
}

// VEC consecutive elements as they are stored (16 or 32 bytes where VEC = 8),
// and their values.  The loads are volatile, and the kernels that add rows state
// how many blocks an SM is to hold, so that the loads stay together: left to
// itself the compiler puts each next to its use, to save registers, and the
// memory's latency is paid for every one (chunks of 32 rows of 768: 39 us).
template <int VEC, bool kF32>
struct Piece {
  static constexpr int kWords = VEC == 1 ? 1 : kF32 ? 8 : 4;
  uint32_t w[kWords];

  MOE_DEV void load(const void* p, size_t i) {
    const uint8_t* q = static_cast<const uint8_t*>(p) + i * (kF32 ? 4 : 2);
    if constexpr (VEC == 1 && kF32) {
      asm volatile("ld.global.b32 %0, [%1];" : "=r"(w[0]) : "l"(q));
    } else if constexpr (VEC == 1) {
      uint16_t h;
      asm volatile("ld.global.b16 %0, [%1];" : "=h"(h) : "l"(q));
      w[0] = static_cast<uint32_t>(h) << 16;
    } else if constexpr (kF32) {
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(q));
    } else {
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(q));
    }
  }
  MOE_DEV float operator[](int e) const {
    if constexpr (VEC == 1 || kF32) return __uint_as_float(w[e]);
    else return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
  }
};

// 8 floats as one store of 32 bytes: as two of 16, each touching half of every
// sector, a fill of 1 GB took 290 us instead of 145.
template <int VEC, bool kF32>
MOE_DEV void store_vec(void* p, size_t i, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    if (kF32) static_cast<float*>(p)[i] = v[0];
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[0]);
  } else if constexpr (kF32) {
    float* q = static_cast<float*>(p) + i;
    if (reinterpret_cast<uintptr_t>(q) & 31) {
      *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                   "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                   : "memory");
    }
  } else {
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i),
           make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
  }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
constexpr int kFwdVecs = 4;  // pieces of a lane

template <int VEC, bool kTabF32, bool kOutF32>
__global__ void __launch_bounds__(256) embedding_kernel(EmbeddingArgs a, int lanes_log2) {
  const int lanes = 1 << lanes_log2;
  const size_t row = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) >> lanes_log2;
  const int lane = threadIdx.x & (lanes - 1);
  if (row >= static_cast<size_t>(a.T)) return;
  const long long id = load_id(a.ids, a.ids64, row);
  const bool known = id >= 0 && id < a.V;
  const int nv = a.D / VEC;
  const size_t src = known ? static_cast<size_t>(id) * a.D : 0, dst = row * a.D;
  for (int v0 = lane; v0 < nv; v0 += kFwdVecs * lanes) {
    Piece<VEC, kTabF32> v[kFwdVecs];
#pragma unroll
    for (int i = 0; i < kFwdVecs; ++i)
      if (v0 + i * lanes < nv) v[i].load(a.table, src + static_cast<size_t>(v0 + i * lanes) * VEC);
#pragma unroll
    for (int i = 0; i < kFwdVecs; ++i)
      if (v0 + i * lanes < nv) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = known ? v[i][j] * a.scale : 0.f;
        store_vec<VEC, kOutF32>(a.out, dst + static_cast<size_t>(v0 + i * lanes) * VEC, o);
      }
  }
}

template <int VEC>
cudaError_t launch_fwd(const EmbeddingArgs& a, cudaStream_t s) {
  // lanes a row: as few as leave each with kFwdVecs pieces, down to a quarter
  // of that where the rows alone do not fill the device
  const int nv = a.D / VEC, per = a.T >= 4096 ? kFwdVecs : 1;
  int l = 0;
  while (l < 8 && (per << l) < nv) ++l;
  const dim3 grid(static_cast<unsigned>(((static_cast<size_t>(a.T) << l) + 255) / 256));
  auto* k = a.table_fp32 ? (a.out_fp32 ? embedding_kernel<VEC, true, true> : embedding_kernel<VEC, true, false>)
                         : (a.out_fp32 ? embedding_kernel<VEC, false, true> : embedding_kernel<VEC, false, false>);
  return launch_kernel(k, grid, dim3(256), 0, s, false, a, l);
}

// ---------------------------------------------------------------------------
// Sort by id
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 512;
constexpr int kHeld = 8;  // rounds of 32 tokens that a warp keeps in registers

constexpr int kMaxCluster = 16;        // most blocks that sort a short list together
constexpr int kShortBlock = kSortThreads * kHeld;
constexpr int kShortList = kMaxCluster * kShortBlock;  // (its positions fit in 16 bits)
constexpr int kPortable = 4096;  // longest list of a cluster that every device holds

struct SortPlan {
  int passes, bits;       // of a pass
  int block, blocks;      // tokens of a block
  int cluster;            // blocks of a short list's cluster, 0 for a launch a pass
  int chunk, chunks;      // aligned runs of sorted tokens
};

// large_clusters: whether the device holds a cluster of kMaxCluster, more than the
// portable 8.  Without, lists past kPortable take a launch a pass.
SortPlan sort_plan(int T, int V, bool large_clusters) {
  SortPlan p = {};
  int b = 1;
  while ((V >> b) != 0) ++b;  // the keys are 0 .. V (V: no row)
  p.passes = (b + 8) / 9;
  p.bits = (b + p.passes - 1) / p.passes;
  if (T <= (large_clusters ? kShortList : kPortable)) {
    // (8000 tokens into 5001 rows of 64: 16 blocks 22.3 us a call, 8 22.6, 4 24.2; 32768
    // into 50001 rows of 768, tied: 16 69, 8 76)
    p.cluster = T <= 512 ? 1 : T <= kPortable ? 4 : kMaxCluster;
    p.block = kSortThreads;
    while (p.block * p.cluster < T) p.block *= 2;
  } else {
    p.block = 2048;
    while (p.block < 32768 && (T + p.block - 1) / p.block > 128) p.block *= 2;
  }
  p.blocks = (T + p.block - 1) / p.block;
  p.chunk = 32;
  while (p.chunk < 1024 && static_cast<long long>(p.chunk) * p.chunk * 16 < T) p.chunk *= 2;
  p.chunks = T > 2048 ? T / p.chunk : 0;  // a short list's long runs need no sums beforehand
  return p;
}

struct SortArgs {
  const void* ids;
  int ids64;
  int T, V;
  int block, blocks, bits, log2_block;
  uint32_t* hist;           // [passes, blocks, 1 << bits]
  const uint32_t* key_in;   // nullptr: from ids
  const uint32_t* tok_in;
  uint32_t* key_out;
  uint32_t* tok_out;
  uint32_t* lists[4];       // keys and tokens, twice
  int pass, passes;
  uint32_t* n_long;         // set to 0
};

MOE_DEV uint32_t sort_key(const SortArgs& a, int i) {
  if (a.key_in) return __ldcg(a.key_in + i);
  const long long id = load_id(a.ids, a.ids64, i);
  return id >= 0 && id < a.V ? static_cast<uint32_t>(id) : static_cast<uint32_t>(a.V);
}

// The first pass's histogram of block `block`, and zeros for the later passes'.
MOE_DEV void first_histogram(const SortArgs& a, int block, uint32_t (&h)[kMaxBins]) {
  const int bins = 1 << a.bits;
  for (int d = threadIdx.x; d < bins; d += kSortThreads) h[d] = 0;
  __syncthreads();
  const int i0 = block * a.block, i1 = min(a.T, i0 + a.block);
#pragma unroll 4
  for (int i = i0 + threadIdx.x; i < i1; i += kSortThreads) atomicAdd(&h[sort_key(a, i) & (bins - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) {
    a.hist[static_cast<size_t>(block) * bins + d] = h[d];
    for (int q = 1; q < a.passes; ++q) a.hist[(static_cast<size_t>(q) * a.blocks + block) * bins + d] = 0;
  }
}

struct SortSmem {
  uint16_t cnt[kSortWarps][kMaxBins];
  uint32_t base[kMaxBins];
  uint32_t warp_total[kSortWarps];
};

// One stable pass over block `block`: its warps take its tokens in order, 32 at
// a time.  Lists and histograms that other blocks have written are read from L2.
MOE_DEV void sort_pass(const SortArgs& a, int block, SortSmem& sm) {
  auto& cnt = sm.cnt;
  auto& base = sm.base;
  auto& warp_total = sm.warp_total;
  const int bins = 1 << a.bits, shift = a.pass * a.bits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_warp = a.block / kSortWarps;
  const int w0 = min(a.T, block * a.block + warp * per_warp), w1 = min(min(a.T, (block + 1) * a.block), w0 + per_warp);
  // the first kHeld rounds' tokens stay in registers
  uint32_t key[kHeld], tok[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = w0 + 32 * k + lane;
    key[k] = i < w1 ? sort_key(a, i) : 0u;
    tok[k] = i < w1 && a.key_in ? __ldcg(a.tok_in + i) : static_cast<uint32_t>(i);
  }
  for (int i = threadIdx.x; i < kSortWarps * kMaxBins / 2; i += kSortThreads)
    reinterpret_cast<uint32_t*>(&cnt[0][0])[i] = 0;
  // where the block's tokens of each digit begin: all smaller digits, then the
  // same digit in earlier blocks
  const uint32_t* hist = a.hist + static_cast<size_t>(a.pass) * a.blocks * bins;
  static_assert(kMaxBins <= kSortThreads);
  uint32_t total = 0, before = 0;
  if (threadIdx.x < bins) {
#pragma unroll 8
    for (int b = 0; b < a.blocks; ++b) {
      const uint32_t v = __ldcg(hist + static_cast<size_t>(b) * bins + threadIdx.x);
      total += v;
      if (b < block) before += v;
    }
  }
  uint32_t incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  uint32_t run = incl - total;
  for (int w = 0; w < warp; ++w) run += warp_total[w];
  if (threadIdx.x < bins) base[threadIdx.x] = run + before;
  const int rounds = (max(w1 - w0, 0) + 31) / 32;
  auto count = [&](int r, uint32_t k) {
    const bool there = w0 + 32 * r + lane < w1;
    const uint32_t d = there ? (k >> shift) & (bins - 1) : 0xffffffffu;
    const uint32_t peers = __match_any_sync(0xffffffffu, d);
    if (there && __ffs(peers) - 1 == lane) cnt[warp][d] += static_cast<uint16_t>(__popc(peers));
    __syncwarp();
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r < rounds) count(r, key[r]);
  for (int r = kHeld; r < rounds; ++r) {
    const int i = w0 + 32 * r + lane;
    count(r, i < w1 ? sort_key(a, i) : 0u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) {
    uint16_t sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint16_t c = cnt[w][d];
      cnt[w][d] = sum;
      sum += c;
    }
  }
  __syncthreads();
  auto place = [&](int r, uint32_t k, uint32_t t) {
    const bool there = w0 + 32 * r + lane < w1;
    const uint32_t d = there ? (k >> shift) & (bins - 1) : 0xffffffffu;
    const uint32_t peers = __match_any_sync(0xffffffffu, d);
    if (there) {
      const uint32_t pos = base[d] + cnt[warp][d] + __popc(peers & ((1u << lane) - 1));
      a.key_out[pos] = k;
      a.tok_out[pos] = t;
      if (a.pass + 1 < a.passes)
        atomicAdd(&a.hist[(static_cast<size_t>(a.pass + 1) * a.blocks + pos / a.block) * bins +
                          ((k >> (shift + a.bits)) & (bins - 1))],
                  1u);
    }
    __syncwarp();
    if (there && __ffs(peers) - 1 == lane) cnt[warp][d] += static_cast<uint16_t>(__popc(peers));
    __syncwarp();
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r < rounds) place(r, key[r], tok[r]);
  for (int r = kHeld; r < rounds; ++r) {
    const int i = w0 + 32 * r + lane;
    place(r, i < w1 ? sort_key(a, i) : 0u, i < w1 && a.key_in ? __ldcg(a.tok_in + i) : static_cast<uint32_t>(i));
  }
}

// Long lists: a launch for the histograms and one for each pass.
__global__ void __launch_bounds__(kSortThreads) embedding_hist_kernel(SortArgs a) {
  __shared__ uint32_t h[kMaxBins];
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_long = 0;
  first_histogram(a, blockIdx.x, h);
}

__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(SortArgs a) {
  __shared__ SortSmem sm;
  griddep_launch_dependents();
  griddep_wait();
  sort_pass(a, blockIdx.x, sm);
}

// Short lists: the whole sort by one cluster, on chip.  Block b holds sorted
// positions [b << log2_block, ...) of the list in shared memory; a warp takes its
// tokens into registers, the blocks see one another's histograms, and every
// token goes to its place in some block's memory, in the last pass to the lists.
// It runs beside a fill that keeps the memory busy: with lists and histograms in
// global memory 32768 tokens took 52 us there, 31 alone; on chip, by 8 blocks, 38
// and 27, by 16 19 alone.
struct ShortSmem {
  uint32_t key[kShortBlock];
  uint16_t tok[kShortBlock];
  uint16_t cnt[kSortWarps][kMaxBins];
  uint32_t hist[kMaxBins];
  uint32_t base[kMaxBins];
  uint32_t warp_total[kSortWarps];
};

MOE_DEV uint32_t load_remote(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_cta(smem_u32(p), rank)) : "memory");
  return v;
}

template <int kCluster>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortThreads) embedding_sort_short_kernel(SortArgs a) {
  __shared__ ShortSmem sm;
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_long = 0;
  const int bins = 1 << a.bits, block = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_warp = a.block / kSortWarps;                      // a multiple of 32
  const int here = max(0, min(a.block, a.T - block * a.block));   // tokens of this block
  const int w0 = warp * per_warp, rounds = max(0, (min(here - w0, per_warp) + 31) / 32);
  const uint32_t below = (1u << lane) - 1;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    uint32_t key[kHeld], tok[kHeld], d[kHeld], peers[kHeld];
#pragma unroll
    for (int r = 0; r < kHeld; ++r) {
      const int i = w0 + 32 * r + lane;
      const bool there = r < rounds && i < here;
      key[r] = !there ? 0u : pass ? sm.key[i] : sort_key(a, block * a.block + i);
      tok[r] = !there ? 0u : pass ? sm.tok[i] : static_cast<uint32_t>(block * a.block + i);
      d[r] = there ? (key[r] >> shift) & (bins - 1) : 0xffffffffu;
    }
    for (int i = threadIdx.x; i < kSortWarps * kMaxBins / 2; i += kSortThreads)
      reinterpret_cast<uint32_t*>(&sm.cnt[0][0])[i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kHeld; ++r) {
      if (r >= rounds) break;
      peers[r] = __match_any_sync(0xffffffffu, d[r]);
      const bool first = d[r] != 0xffffffffu && (peers[r] & below) == 0;
      // where this round's tokens of the digit go among the warp's
      uint16_t before = 0;
      if (first) {
        before = sm.cnt[warp][d[r]];
        sm.cnt[warp][d[r]] = static_cast<uint16_t>(before + __popc(peers[r]));
      }
      // (in the lower half the digit, in the upper the place)
      const uint32_t lead = __shfl_sync(0xffffffffu, static_cast<uint32_t>(before), __ffs(peers[r]) - 1);
      d[r] = d[r] == 0xffffffffu ? d[r] : d[r] | (lead + __popc(peers[r] & below)) << 16;
      __syncwarp();
    }
    __syncthreads();
    // the block's histogram, and each warp's place in it
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
      uint32_t sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = sm.cnt[w][b];
        sm.cnt[w][b] = static_cast<uint16_t>(sum);
        sum += c;
      }
      sm.hist[b] = sum;
    }
    cluster_sync_all();  // and every block has its tokens in registers
    uint32_t total = 0, before = 0;
    if (threadIdx.x < bins) {
#pragma unroll
      for (int b = 0; b < kCluster; ++b) {
        const uint32_t v = load_remote(&sm.hist[threadIdx.x], b);
        total += v;
        if (b < block) before += v;
      }
    }
    uint32_t incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sm.warp_total[warp] = incl;
    __syncthreads();
    uint32_t run = incl - total;
    for (int w = 0; w < warp; ++w) run += sm.warp_total[w];
    if (threadIdx.x < bins) sm.base[threadIdx.x] = run + before;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kHeld; ++r) {
      if (r >= rounds || d[r] == 0xffffffffu) continue;
      const uint32_t digit = d[r] & 0xffffu, pos = sm.base[digit] + sm.cnt[warp][digit] + (d[r] >> 16);
      if (pass + 1 == a.passes) {
        a.lists[0][pos] = key[r];
        a.lists[1][pos] = tok[r];
      } else {
        const uint32_t to = pos >> a.log2_block, at = pos & (a.block - 1);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_cta(smem_u32(&sm.key[at]), to)), "r"(key[r]) : "memory");
        asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(map_to_cta(smem_u32(&sm.tok[at]), to)),
                     "h"(static_cast<uint16_t>(tok[r]))
                     : "memory");
      }
    }
    cluster_sync_all();  // the tokens have arrived; nobody reads this block's histogram any more
  }
}

// Every row of the table: zeros, or `add`.  It runs beside the sort before it
// and ends after it, so that what waits for this kernel may read both.  (In one
// launch with the sort's cluster, as clusters too, it filled at 5.5 TB/s instead
// of 7.5: clusters of 8 leave part of the SMs empty.)
constexpr int kFillThreads = 512;
constexpr int kFillEach = 4;     // pieces of 8 that a thread has in flight
constexpr int kFillBlocks = 64;  // of an SM, one after the other (4: 160 us for 1 GB, 64: 142)

__global__ void __launch_bounds__(kFillThreads) embedding_fill_kernel(float* out, const uint16_t* add, size_t n) {
  griddep_launch_dependents();
  const size_t pieces = n / 8, step = static_cast<size_t>(kFillThreads) * kFillEach;
  for (size_t p = blockIdx.x * step; p < pieces; p += gridDim.x * step) {
    Piece<8, false> v[kFillEach] = {};
    if (add) {
#pragma unroll
      for (int i = 0; i < kFillEach; ++i)
        v[i].load(add, min(p + static_cast<size_t>(i) * kFillThreads + threadIdx.x, pieces - 1) * 8);
    }
#pragma unroll
    for (int i = 0; i < kFillEach; ++i) {
      const size_t q = p + static_cast<size_t>(i) * kFillThreads + threadIdx.x;
      if (q < pieces) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = v[i][e];
        store_vec<8, true>(out, q * 8, o);
      }
    }
  }
  if (blockIdx.x == 0) {  // the last few elements
    const size_t i = pieces * 8 + threadIdx.x;
    if (i < n) out[i] = add ? __uint_as_float(static_cast<uint32_t>(add[i]) << 16) : 0.f;
    griddep_wait();  // (a block that waits keeps its place on the SM: one is enough)
  }
}

// ---------------------------------------------------------------------------
// Sums of rows
// ---------------------------------------------------------------------------
struct SumArgs {
  const void* d_out;
  const void* add;         // bf16 or nullptr
  const uint32_t* key;     // sorted
  const uint32_t* tok;
  float* part;             // [chunks, D]
  float* d_table;
  float scale;
  int T, V, D, chunk, chunks;
  int window_blocks, chunk_blocks;
  int2* long_runs;         // with chunks: [start, end) of each
  uint32_t* n_long;
};

constexpr int kWindow = 4;     // sorted tokens of a warp
constexpr int kSumWarps = 8;
constexpr int kSumBlocks = 2;  // of an SM
constexpr int kLong = 16;      // tokens past its window that a warp adds alone

// A warp's columns of one turn: kVecs pieces of a lane, kAhead rows in flight.
template <int VEC, bool kF32>
struct Shape {
  static constexpr int kVecs = VEC == 1 ? 8 : kF32 ? 2 : 3;
  static constexpr int kColumns = 32 * kVecs * VEC;
};
template <int VEC, bool kF32, int kVecs>
constexpr int kAhead = VEC == 1 || kVecs * Piece<VEC, kF32>::kWords <= 16 ? 4 : 2;  // at most 64 registers

// A lane's pieces of one row; lanes past the last column read another's (a load
// under a condition would be waited for on the spot).
template <int VEC, bool kF32, int N>
MOE_DEV void load_row(const void* src, uint32_t row, int D, int v0, int nv, Piece<VEC, kF32> (&v)[N]) {
  const size_t at = static_cast<size_t>(row) * D;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i].load(src, at + static_cast<size_t>(min(v0 + 32 * i, nv - 1)) * VEC);
}

// acc += rows row(0) .. row(n - 1) of `src`, in that order, R in flight (the
// last of them again where there are fewer left).
template <int VEC, bool kF32, int kVecs, typename Index>
MOE_DEV void add_rows(const void* src, int D, int v0, int nv, int n, Index row, float (&acc)[kVecs][VEC]) {
  constexpr int R = kAhead<VEC, kF32, kVecs>;
#pragma unroll 1
  for (int j = 0; j < n; j += R) {
    Piece<VEC, kF32> v[R][kVecs];
#pragma unroll
    for (int r = 0; r < R; ++r) load_row(src, row(min(j + r, n - 1)), D, v0, nv, v[r]);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (j + r < n)
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[i][e] += v[r][i][e];
  }
}

// Sum of an aligned run of `chunk` sorted tokens, where it has one id: warp
// `job` of chunks x turns of columns.
template <int VEC, bool kF32>
MOE_DEV void sum_chunk(const SumArgs& a, int job) {
  constexpr int kVecs = Shape<VEC, kF32>::kVecs;
  const int c = job % a.chunks, lane = threadIdx.x & 31;
  const int nv = a.D / VEC, v0 = job / a.chunks * 32 * kVecs + lane;
  if (v0 - lane >= nv) return;
  const size_t p0 = static_cast<size_t>(c) * a.chunk;
  const uint32_t k = a.key[p0];
  if (k != a.key[p0 + a.chunk - 1] || k >= static_cast<uint32_t>(a.V)) return;
  float acc[kVecs][VEC] = {};
  for (int j = 0; j < a.chunk; j += 32) {
    const uint32_t tok = a.tok[p0 + j + lane];
    add_rows<VEC, kF32>(a.d_out, a.D, v0, nv, 32, [&](int r) { return __shfl_sync(0xffffffffu, tok, r); }, acc);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    if (v0 + 32 * i < nv)
      store_vec<VEC, true>(a.part, static_cast<size_t>(c) * a.D + static_cast<size_t>(v0 + 32 * i) * VEC, acc[i]);
}

// First sorted position from lo on whose key is more than k (whole warp).
MOE_DEV int end_of(const uint32_t* key, int lo, int T, uint32_t k) {
  const int lane = threadIdx.x & 31;
  const int near = __popc(__ballot_sync(0xffffffffu, lo + lane < T && key[min(lo + lane, T - 1)] <= k));
  if (near < 32) return lo + near;
  lo += 32;
  int hi = T;  // the answer lies in [lo, hi]
  while (hi - lo > 32) {
    const int at = lo + static_cast<int>(static_cast<long long>(hi - lo) * (lane + 1) / 33);
    const uint32_t le = __ballot_sync(0xffffffffu, key[at] <= k);
    const int n = __popc(le);  // the probes ascend, so the first n are at most k
    const int left = n == 0 ? lo : __shfl_sync(0xffffffffu, at, n - 1) + 1;
    const int right = n == 32 ? hi : __shfl_sync(0xffffffffu, at, n & 31);
    lo = left;
    hi = right;
  }
  return lo + __popc(__ballot_sync(0xffffffffu, lo + lane < hi && key[lo + lane] <= k));
}

// (`add` is read again, not added to what the row was filled with by an atomic of
// the memory: that takes subnormal numbers for zeros.)
template <int VEC, int kVecs>
MOE_DEV void write_row(const SumArgs& a, uint32_t v, int v0, int nv, const float (&acc)[kVecs][VEC]) {
  const size_t row = static_cast<size_t>(v) * a.D;
  Piece<VEC, false> with[kVecs] = {};
  if (a.add) load_row(a.add, v, a.D, v0, nv, with);
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    if (v0 + 32 * i < nv) {
      float o[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        o[e] = a.scale * acc[i][e];
        if (a.add) o[e] = __fadd_rn(with[i][e], o[e]);
      }
      store_vec<VEC, true>(a.d_table, row + static_cast<size_t>(v0 + 32 * i) * VEC, o);
    }
}

// One turn of columns of the long run [start, end), by the whole block: rows up
// to the first chunk that lies inside, the chunks' sums, the rows behind them;
// every warp takes a share.
template <int VEC, bool kF32>
MOE_DEV void add_long_run(const SumArgs& a, int start, int end, int turn,
                          float (&red)[kSumWarps][Shape<VEC, kF32>::kColumns]) {
  constexpr int kVecs = Shape<VEC, kF32>::kVecs, kColumns = Shape<VEC, kF32>::kColumns;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nv = a.D / VEC;
  const int c0 = (start + a.chunk - 1) / a.chunk, c1 = a.chunks ? max(c0, end / a.chunk) : c0;
  const int head = c0 < c1 ? c0 * a.chunk - start : end - start;
  const int tail = c0 < c1 ? c1 * a.chunk : end;
  auto share = [&](int n, int i) { return static_cast<int>(static_cast<long long>(n) * i / kSumWarps); };
  const int col = turn * 32 * kVecs, v0 = col + lane;
  float acc[kVecs][VEC] = {};
  const int h0 = start + share(head, warp), h1 = start + share(head, warp + 1);
  add_rows<VEC, kF32>(a.d_out, a.D, v0, nv, h1 - h0, [&](int r) { return a.tok[h0 + r]; }, acc);
  const int m0 = c0 + share(c1 - c0, warp), m1 = c0 + share(c1 - c0, warp + 1);
  add_rows<VEC, true>(a.part, a.D, v0, nv, m1 - m0, [&](int r) { return m0 + r; }, acc);
  const int t0 = tail + share(end - tail, warp), t1 = tail + share(end - tail, warp + 1);
  add_rows<VEC, kF32>(a.d_out, a.D, v0, nv, t1 - t0, [&](int r) { return a.tok[t0 + r]; }, acc);
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) red[warp][(32 * i + lane) * VEC + e] = acc[i][e];
  __syncthreads();
  const size_t dst = static_cast<size_t>(a.key[start]) * a.D;
  for (int c = threadIdx.x; c < kColumns; c += 32 * kSumWarps) {
    const int column = col * VEC + c;
    if (column >= a.D) break;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kSumWarps; ++i) sum += red[i][c];
    Piece<1, false> with = {};
    if (a.add) with.load(a.add, dst + column);
    a.d_table[dst + column] = a.add ? __fadd_rn(with[0], a.scale * sum) : a.scale * sum;
  }
  __syncthreads();
}

// The listed long runs, a turn of columns at a time.  (A block for each block of
// windows, most of them with nothing to do: 187 us a call of 200000 x 768 into
// 50001 rows instead of 174.)
template <int VEC, bool kF32>
__global__ void __launch_bounds__(32 * kSumWarps, kSumBlocks) embedding_long_kernel(SumArgs a, int turns) {
  __shared__ float red[kSumWarps][Shape<VEC, kF32>::kColumns];
  griddep_wait();
  const int n = static_cast<int>(*a.n_long) * turns;
#pragma unroll 1
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int2 run = a.long_runs[i / turns];
    add_long_run<VEC, kF32>(a, run.x, run.y, i % turns, red);
  }
}

// A warp a window of sorted tokens: the rows whose tokens begin there.  The
// first blocks sum the chunks, which takes longest (as the last ones: 76 us a call
// of 32768 x 768 into 50001 rows instead of 70); the long runs, listed here, wait
// for those.
template <int VEC, bool kF32>
__global__ void __launch_bounds__(32 * kSumWarps, kSumBlocks) embedding_rows_kernel(SumArgs a) {
  constexpr int kVecs = Shape<VEC, kF32>::kVecs, R = kAhead<VEC, kF32, kVecs>;
  static_assert(kWindow % R == 0);
  __shared__ float red[kSumWarps][Shape<VEC, kF32>::kColumns];
  __shared__ int2 runs[kSumWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int block = static_cast<int>(blockIdx.x) - a.chunk_blocks;
  if (block < 0) {
    if (blockIdx.y == 0) sum_chunk<VEC, kF32>(a, blockIdx.x * kSumWarps + (threadIdx.x >> 5));
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int p0 = (block * kSumWarps + warp) * kWindow;
  const int nv = a.D / VEC, turns = (nv + 32 * kVecs - 1) / (32 * kVecs);
  const int turn0 = turns * blockIdx.y / gridDim.y, turn1 = turns * (blockIdx.y + 1) / gridDim.y;
  const uint32_t none = static_cast<uint32_t>(a.V);  // tokens without a row, sorted to the end, and what lies past it
  const int at = p0 - 1 + lane;                      // lane 0 sees the token before the window
  const uint32_t k = at < 0 ? 0xffffffffu : at < a.T ? a.key[at] : none;
  const uint32_t my_tok = a.tok[min(max(at, 0), a.T - 1)];
  const uint32_t k_before = __shfl_up_sync(0xffffffffu, k, 1);
  const uint32_t begins = __ballot_sync(0xffffffffu, lane >= 1 && lane <= kWindow && k != k_before && k < none) >> 1;
  // tokens of the last run behind the window, as far as the lanes see
  const uint32_t last = __shfl_sync(0xffffffffu, k, kWindow);
  const int len_past = __popc(__ballot_sync(0xffffffffu, begins != 0 && lane > kWindow && k == last && last < none));
  static_assert(kWindow + 1 + kLong < 32);
  const bool is_long = len_past > kLong;
  if (lane == 0) runs[warp] = make_int2(-1, -1);
  if (begins) {
    const int first = __ffs(begins) - 1;
    // past the window, a run too long for this warp, or the tokens without a row
    const uint32_t rows = __ballot_sync(0xffffffffu, lane >= 1 && lane <= kWindow && k < none) >> 1;
    const int stop = is_long ? 31 - __clz(begins) : 32 - __clz(rows);
#pragma unroll 1
    for (int turn = turn0; turn < turn1; ++turn) {
      const int v0 = turn * 32 * kVecs + lane;
      float acc[kVecs][VEC] = {};
#pragma unroll 1
      for (int b = 0; b < stop; b += R) {
        if (b + R <= first) continue;
        Piece<VEC, kF32> x[R][kVecs];
#pragma unroll
        for (int r = 0; r < R; ++r) load_row(a.d_out, __shfl_sync(0xffffffffu, my_tok, b + r + 1), a.D, v0, nv, x[r]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int j = b + r;
          if (j < first || j >= stop) continue;
          const bool begin = begins >> j & 1;
#pragma unroll
          for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[i][e] = begin ? x[r][i][e] : acc[i][e] + x[r][i][e];
          if (j + 1 < stop && !(begins >> (j + 1) & 1)) continue;
          if (j + 1 == kWindow)
            add_rows<VEC, kF32>(a.d_out, a.D, v0, nv, len_past,
                                [&](int q) { return __shfl_sync(0xffffffffu, my_tok, kWindow + 1 + q); }, acc);
          write_row(a, __shfl_sync(0xffffffffu, k, j + 1), v0, nv, acc);
        }
      }
    }
  }
  if (is_long && !(a.chunks && blockIdx.y > 0)) {
    const int end = end_of(a.key, p0 + kWindow, a.T, last);
    const int2 run = make_int2(p0 + 31 - __clz(begins), end);
    // (any order will do: each run is added by itself)
    if (lane == 0 && a.chunks) a.long_runs[atomicAdd(a.n_long, 1u)] = run;
    else if (lane == 0) runs[warp] = run;
  }
  if (a.chunks) return;
  __syncthreads();
#pragma unroll 1
  for (int w = 0; w < kSumWarps; ++w)
    if (runs[w].x >= 0)
#pragma unroll 1
      for (int turn = turn0; turn < turn1; ++turn) add_long_run<VEC, kF32>(a, runs[w].x, runs[w].y, turn, red);
}

// fp32 rows are read 32 bytes at a time.
bool on32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

size_t padded(size_t n) { return (n + 255) / 256 * 256; }

template <int VEC, bool kF32>
cudaError_t launch_sums(SumArgs a, cudaStream_t s) {
  const int turns = (a.D + Shape<VEC, kF32>::kColumns - 1) / Shape<VEC, kF32>::kColumns;
  a.chunk_blocks = (a.chunks * turns + kSumWarps - 1) / kSumWarps;
  const int fit = kSumBlocks * std::max(current_device_sms(), 1);
  // few tokens: a window's columns are shared among blocks (562 x 3346 into 371 rows: 22
  // us a call, with one block a window 51; 8000 x 1025 into 20000: 43 and 50)
  const int share = std::min(turns, (fit + a.window_blocks - 1) / a.window_blocks);
  const cudaError_t e = launch_kernel(embedding_rows_kernel<VEC, kF32>, dim3(a.window_blocks + a.chunk_blocks, share),
                                      dim3(32 * kSumWarps), 0, s, true, a);
  if (e != cudaSuccess || !a.chunks) return e;
  return launch_kernel(embedding_long_kernel<VEC, kF32>, dim3(fit), dim3(32 * kSumWarps), 0, s, true, a, turns);
}

std::mutex g_mu;
int g_large_clusters[64];  // of a device: 0 not asked yet, 1 held, -1 not held

// Clusters of 16 have to be allowed and found to fit, once on each device.
cudaError_t large_clusters(bool* held) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mu);
  int& known = g_large_clusters[dev];
  if (known == 0) {
    auto* k = embedding_sort_short_kernel<kMaxCluster>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMaxCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCluster);
    cfg.blockDim = dim3(kSortThreads);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int fit = 0;
    const bool ok = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&fit, k, &cfg) == cudaSuccess && fit > 0;
    if (!ok) cudaGetLastError();  // a refusal is an answer, not this call's error
    known = ok ? 1 : -1;
  }
  *held = known == 1;
  return cudaSuccess;
}

cudaError_t launch_sort_short(const SortArgs& q, int cluster, cudaStream_t s) {
  auto* k = cluster == 1   ? embedding_sort_short_kernel<1>
            : cluster == 4 ? embedding_sort_short_kernel<4>
                           : embedding_sort_short_kernel<kMaxCluster>;
  return launch_kernel(k, dim3(cluster), dim3(kSortThreads), 0, s, false, q);
}

// (a list that a cluster of 16 may sort has room for the other way too: the size
// depends on no device)
size_t hist_bytes(int T, int V) {
  const SortPlan p = sort_plan(T, V, false);
  return p.cluster ? 0 : static_cast<size_t>(p.passes) * p.blocks * (sizeof(uint32_t) << p.bits);
}

int window_blocks(int T) { return (T + kSumWarps * kWindow - 1) / (kSumWarps * kWindow); }

// Long runs of T sorted tokens at most, each with a token in its window.
size_t most_long(int T) { return static_cast<size_t>(T) / (kLong + 2) + 1; }

}  // namespace

cudaError_t launch_embedding(const EmbeddingArgs& a, cudaStream_t s) {
  return a.D % 8 == 0 && (!a.table_fp32 || on32(a.table)) ? launch_fwd<8>(a, s) : launch_fwd<1>(a, s);
}

size_t embedding_bwd_scratch_bytes(int T, int V, int D) {
  const SortPlan p = sort_plan(T, V, true);
  return padded(hist_bytes(T, V)) +
         4 * padded(static_cast<size_t>(T) * sizeof(uint32_t)) + padded(static_cast<size_t>(p.chunks) * D * sizeof(float)) +
         padded(sizeof(uint32_t)) + padded(p.chunks ? most_long(T) * sizeof(int2) : 0);
}

cudaError_t launch_embedding_bwd(const EmbeddingBwdArgs& a, void* scratch, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  bool large = false;
  if (a.T > kPortable && a.T <= kShortList && !a.by_passes && (e = large_clusters(&large)) != cudaSuccess) return e;
  const SortPlan p = sort_plan(a.T, a.V, large);
  uint8_t* at = static_cast<uint8_t*>(scratch);
  auto take = [&](size_t bytes) {
    uint8_t* r = at;
    at += padded(bytes);
    return r;
  };
  SortArgs q = {};
  q.ids = a.ids;
  q.ids64 = a.ids64;
  q.T = a.T;
  q.V = a.V;
  q.block = p.block;
  q.blocks = p.blocks;
  q.bits = p.bits;
  while ((1 << q.log2_block) < p.block) ++q.log2_block;
  q.passes = p.passes;
  q.hist = reinterpret_cast<uint32_t*>(take(hist_bytes(a.T, a.V)));
  for (auto& l : q.lists) l = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(a.T) * sizeof(uint32_t)));
  float* part = reinterpret_cast<float*>(take(static_cast<size_t>(p.chunks) * a.D * sizeof(float)));
  q.n_long = reinterpret_cast<uint32_t*>(take(sizeof(uint32_t)));
  int2* long_runs = reinterpret_cast<int2*>(take(p.chunks ? most_long(a.T) * sizeof(int2) : 0));
  if (a.T > 0 && p.cluster) {
    e = launch_sort_short(q, p.cluster, s);
  } else if (a.T > 0) {
    e = launch_kernel(embedding_hist_kernel, dim3(p.blocks), dim3(kSortThreads), 0, s, false, q);
    for (q.pass = 0; q.pass < p.passes && e == cudaSuccess; ++q.pass) {
      q.key_out = q.lists[2 * (q.pass & 1)];
      q.tok_out = q.lists[2 * (q.pass & 1) + 1];
      e = launch_kernel(embedding_sort_kernel, dim3(p.blocks), dim3(kSortThreads), 0, s, true, q);
      q.key_in = q.key_out;
      q.tok_in = q.tok_out;
    }
  }
  if (e != cudaSuccess) return e;
  const size_t n = static_cast<size_t>(a.V) * a.D, per = static_cast<size_t>(kFillThreads) * kFillEach * 8;
  const size_t fit = static_cast<size_t>(kFillBlocks) * std::max(current_device_sms(), 1);
  e = launch_kernel(embedding_fill_kernel, dim3(static_cast<unsigned>(std::min((n + per - 1) / per, fit))), dim3(kFillThreads),
                    0, s, a.T > 0, a.d_table, static_cast<const uint16_t*>(a.add), n);
  if (e != cudaSuccess || a.T == 0) return e;
  const int last = p.cluster ? 0 : (p.passes - 1) & 1;
  const SumArgs m{a.d_out, a.add, q.lists[2 * last], q.lists[2 * last + 1], part, a.d_table, a.scale, a.T, a.V, a.D, p.chunk, p.chunks,
                  window_blocks(a.T), 0, long_runs, q.n_long};
  if (a.D % 8 == 0 && (!a.d_fp32 || on32(a.d_out))) return a.d_fp32 ? launch_sums<8, true>(m, s) : launch_sums<8, false>(m, s);
  return a.d_fp32 ? launch_sums<1, true>(m, s) : launch_sums<1, false>(m, s);
}

}  // namespace moe
