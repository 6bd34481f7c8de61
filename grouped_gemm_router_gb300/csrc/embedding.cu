// Embedding lookup, out[t] = scale table[ids[t]], and its gradient,
// d_table[v] = (add[v] +) scale sum over {t : ids[t] = v} of d_out[t].
//
// Both are bound by memory.  The lookup gives a row to a few lanes, up to four
// 16-byte pieces each.
//
// The gradient sorts the tokens by id (stable radix sort, most of 10 bits a
// pass, so two passes up to a million ids), then a warp a few rows of the table:
// it finds its rows' tokens in the sorted list by a 33-way search, adds their
// gradients in token order in fp32 and writes the row, so that every row is
// written once, in order, and no sum depends on timing.  Frequent tokens would
// leave one warp with thousands of rows to add: aligned runs of `chunk` sorted
// tokens with one id are summed beforehand by warps of their own.
#include <algorithm>

#include "moe_device.cuh"
#include "moe_kernels.cuh"

namespace moe {
namespace {

MOE_DEV long long load_id(const void* p, int is64, size_t i) {
  return is64 ? static_cast<const long long*>(p)[i] : static_cast<const int*>(p)[i];
}

// VEC consecutive elements as they are stored (16 or 32 bytes where VEC = 8),
// and their values.
template <int VEC, bool kF32>
struct Piece {
  static constexpr int kWords = VEC == 1 ? 1 : kF32 ? 8 : 4;
  uint32_t w[kWords];

  MOE_DEV void load(const void* p, size_t i) {
    if constexpr (VEC == 1) {
      w[0] = kF32 ? static_cast<const uint32_t*>(p)[i] : static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16;
    } else {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (kF32 ? 4 : 2));
#pragma unroll
      for (int k = 0; k < kWords / 4; ++k) {
        const uint4 x = q[k];
        w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
      }
    }
  }
  MOE_DEV float operator[](int e) const {
    if constexpr (VEC == 1 || kF32) return __uint_as_float(w[e]);
    else return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
  }
};

template <int VEC, bool kF32>
MOE_DEV void store_vec(void* p, size_t i, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    if (kF32) static_cast<float*>(p)[i] = v[0];
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[0]);
  } else if constexpr (kF32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    __stcs(q, make_float4(v[0], v[1], v[2], v[3]));
    __stcs(q + 1, make_float4(v[4], v[5], v[6], v[7]));
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
constexpr int kMaxBins = 1024;
constexpr int kMaxPasses = 3;

struct SortPlan {
  int passes, bits;       // of a pass
  int block, blocks;      // tokens of a block
  int chunk, chunks;      // aligned runs of sorted tokens
};

SortPlan sort_plan(int T, int V) {
  SortPlan p;
  int b = 1;
  while ((V >> b) != 0) ++b;  // the keys are 0 .. V (V: no row)
  p.passes = b <= 10 ? 1 : b <= 20 ? 2 : 3;
  p.bits = (b + p.passes - 1) / p.passes;
  p.block = 2048;
  while (p.block < 32768 && (T + p.block - 1) / p.block > 128) p.block *= 2;
  p.blocks = (T + p.block - 1) / p.block;
  p.chunk = 32;
  while (p.chunk < 1024 && static_cast<long long>(p.chunk) * p.chunk * 16 < T) p.chunk *= 2;
  p.chunks = T / p.chunk;
  return p;
}

struct SortArgs {
  const void* ids;
  int ids64;
  int T, V;
  int block, blocks, bits;
  uint32_t* hist;           // [passes, blocks, 1 << bits]
  const uint32_t* key_in;   // nullptr: from ids
  const uint32_t* tok_in;
  uint32_t* key_out;
  uint32_t* tok_out;
  int pass, passes;
};

MOE_DEV uint32_t sort_key(const SortArgs& a, int i) {
  if (a.key_in) return a.key_in[i];
  const long long id = load_id(a.ids, a.ids64, i);
  return id >= 0 && id < a.V ? static_cast<uint32_t>(id) : static_cast<uint32_t>(a.V);
}

// The first pass's histograms of the blocks, and zeros for the later passes'.
__global__ void __launch_bounds__(kSortThreads) embedding_hist_kernel(SortArgs a) {
  __shared__ uint32_t h[kMaxBins];
  griddep_launch_dependents();
  const int bins = 1 << a.bits;
  for (int d = threadIdx.x; d < bins; d += kSortThreads) h[d] = 0;
  __syncthreads();
  const int i0 = blockIdx.x * a.block, i1 = min(a.T, i0 + a.block);
  for (int i = i0 + threadIdx.x; i < i1; i += kSortThreads) atomicAdd(&h[sort_key(a, i) & (bins - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) {
    a.hist[static_cast<size_t>(blockIdx.x) * bins + d] = h[d];
    for (int q = 1; q < a.passes; ++q) a.hist[(static_cast<size_t>(q) * a.blocks + blockIdx.x) * bins + d] = 0;
  }
}

// One stable pass: a block's warps take its tokens in order, 32 at a time.
__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(SortArgs a) {
  __shared__ uint16_t cnt[kSortWarps][kMaxBins];
  __shared__ uint32_t base[kMaxBins];
  __shared__ uint32_t warp_total[kSortWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int bins = 1 << a.bits, shift = a.pass * a.bits;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * kMaxBins / 2; i += kSortThreads)
    reinterpret_cast<uint32_t*>(&cnt[0][0])[i] = 0;
  // where the block's tokens of each digit begin: all smaller digits, then the
  // same digit in earlier blocks
  const uint32_t* hist = a.hist + static_cast<size_t>(a.pass) * a.blocks * bins;
  constexpr int kPer = kMaxBins / kSortThreads;
  uint32_t total[kPer], before[kPer], local = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int d = threadIdx.x * kPer + k;
    total[k] = before[k] = 0;
    if (d < bins) {
#pragma unroll 8
      for (int b = 0; b < a.blocks; ++b) {
        const uint32_t v = hist[static_cast<size_t>(b) * bins + d];
        total[k] += v;
        if (b < static_cast<int>(blockIdx.x)) before[k] += v;
      }
    }
    local += total[k];
  }
  uint32_t incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  uint32_t run = incl - local;
  for (int w = 0; w < warp; ++w) run += warp_total[w];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    base[threadIdx.x * kPer + k] = run + before[k];
    run += total[k];
  }
  const int i0 = blockIdx.x * a.block, per_warp = a.block / kSortWarps;
  const int w0 = i0 + warp * per_warp, w1 = min(a.T, w0 + per_warp);
  for (int r = w0; r < w1; r += 32) {
    const bool there = r + lane < w1;
    const uint32_t d = there ? (sort_key(a, r + lane) >> shift) & (bins - 1) : 0xffffffffu;
    const uint32_t peers = __match_any_sync(0xffffffffu, d);
    if (there && __ffs(peers) - 1 == lane) cnt[warp][d] += static_cast<uint16_t>(__popc(peers));
    __syncwarp();
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
  for (int r = w0; r < w1; r += 32) {
    const bool there = r + lane < w1;
    const uint32_t key = there ? sort_key(a, r + lane) : 0;
    const uint32_t d = there ? (key >> shift) & (bins - 1) : 0xffffffffu;
    const uint32_t peers = __match_any_sync(0xffffffffu, d);
    if (there) {
      const uint32_t pos = base[d] + cnt[warp][d] + __popc(peers & ((1u << lane) - 1));
      a.key_out[pos] = key;
      a.tok_out[pos] = a.key_in ? a.tok_in[r + lane] : static_cast<uint32_t>(r + lane);
      if (a.pass + 1 < a.passes)
        atomicAdd(&a.hist[(static_cast<size_t>(a.pass + 1) * a.blocks + pos / a.block) * bins +
                          ((key >> (shift + a.bits)) & (bins - 1))],
                  1u);
    }
    __syncwarp();
    if (there && __ffs(peers) - 1 == lane) cnt[warp][d] += static_cast<uint16_t>(__popc(peers));
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// Sums of rows
// ---------------------------------------------------------------------------
struct SumArgs {
  const void* d_out;
  const void* add;         // bf16
  const uint32_t* key;     // sorted
  const uint32_t* tok;
  float* part;             // [chunks, D]
  float* d_table;
  float scale;
  int T, V, D, chunk, chunks;
};

constexpr int kVecs = 4;     // pieces of a lane
constexpr int kRowsPerWarp = 4;

// acc += rows index(0) .. index(n - 1) of `src`, in that order; kAhead of them
// in flight.
template <int VEC, bool kF32, typename Index>
MOE_DEV void add_rows(const void* src, int D, int v0, int nv, int n, Index index, float (&acc)[kVecs][VEC]) {
  constexpr int kAhead = kF32 ? 2 : 4;
#pragma unroll 1
  for (int j = 0; j < n; j += kAhead) {
    Piece<VEC, kF32> v[kAhead][kVecs];
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      const size_t at = static_cast<size_t>(index(min(j + r, n - 1))) * D;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (j + r < n && v0 + 32 * i < nv) v[r][i].load(src, at + static_cast<size_t>(v0 + 32 * i) * VEC);
        else v[r][i] = {};  // (registers that are written under a condition alone stay live around the loop)
    }
#pragma unroll
    for (int r = 0; r < kAhead; ++r)
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[i][e] += v[r][i][e];
  }
}

// Aligned runs of `chunk` sorted tokens with one id, a warp each.
template <int VEC, bool kF32>
__global__ void __launch_bounds__(256) embedding_chunk_kernel(SumArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (c >= a.chunks) return;
  const size_t p0 = static_cast<size_t>(c) * a.chunk;
  const uint32_t k = a.key[p0];
  if (k != a.key[p0 + a.chunk - 1] || k >= static_cast<uint32_t>(a.V)) return;
  const int nv = a.D / VEC;
#pragma unroll 1
  for (int v0 = lane; v0 < nv; v0 += 32 * kVecs) {
    float acc[kVecs][VEC] = {};
    add_rows<VEC, kF32>(a.d_out, a.D, v0, nv, a.chunk, [&](int j) { return a.tok[p0 + j]; }, acc);
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (v0 + 32 * i < nv)
        store_vec<VEC, true>(a.part, static_cast<size_t>(c) * a.D + static_cast<size_t>(v0 + 32 * i) * VEC, acc[i]);
  }
}

// First sorted position whose key is at least k (whole warp).
MOE_DEV int lower_bound(const uint32_t* key, int T, uint32_t k) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = T;  // the answer lies in [lo, hi]
  while (hi - lo > 32) {
    const int at = lo + static_cast<int>(static_cast<long long>(hi - lo) * (lane + 1) / 33);
    const uint32_t less = __ballot_sync(0xffffffffu, key[at] < k);
    const int n = __popc(less);  // the probes ascend, so the first n are less
    const int left = n == 0 ? lo : __shfl_sync(0xffffffffu, at, n - 1) + 1;
    const int right = n == 32 ? hi : __shfl_sync(0xffffffffu, at, n & 31);
    lo = left;
    hi = right;
  }
  const uint32_t less = __ballot_sync(0xffffffffu, lo + lane < hi && key[lo + lane] < k);
  return lo + __popc(less);
}

template <int VEC, bool kF32>
__global__ void __launch_bounds__(256) embedding_rows_kernel(SumArgs a) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long v_first = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kRowsPerWarp;
  if (v_first >= a.V) return;
  const int v_end = static_cast<int>(min(static_cast<long long>(a.V), v_first + kRowsPerWarp));
  const int nv = a.D / VEC;
  int start = lower_bound(a.key, a.T, static_cast<uint32_t>(v_first));
#pragma unroll 1
  for (int v = static_cast<int>(v_first); v < v_end; ++v) {
    const bool there = start + lane < a.T;
    const uint32_t mine = there ? a.key[start + lane] : 0xffffffffu;
    const uint32_t tok = there ? a.tok[start + lane] : 0u;
    int n = __popc(__ballot_sync(0xffffffffu, mine == static_cast<uint32_t>(v)));
    const bool few = n < 32;
    if (!few) n = lower_bound(a.key, a.T, static_cast<uint32_t>(v) + 1) - start;
    const size_t dst = static_cast<size_t>(v) * a.D;
#pragma unroll 1
    for (int v0 = lane; v0 - lane < nv; v0 += 32 * kVecs) {  // the same turns for every lane
      float acc[kVecs][VEC] = {};
      if (few) {
        add_rows<VEC, kF32>(a.d_out, a.D, v0, nv, n, [&](int j) { return __shfl_sync(0xffffffffu, tok, j); }, acc);
      } else {
        // up to the first chunk that lies inside, the chunks, the rest
        const int end = start + n;
        const int c0 = (start + a.chunk - 1) / a.chunk, c1 = end / a.chunk;
        const int head = c0 < c1 ? c0 * a.chunk - start : n;
        add_rows<VEC, kF32>(a.d_out, a.D, v0, nv, head, [&](int j) { return a.tok[start + j]; }, acc);
        if (c0 < c1) {
          add_rows<VEC, true>(a.part, a.D, v0, nv, c1 - c0, [&](int j) { return c0 + j; }, acc);
          const int tail = c1 * a.chunk;
          add_rows<VEC, kF32>(a.d_out, a.D, v0, nv, end - tail, [&](int j) { return a.tok[tail + j]; }, acc);
        }
      }
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (v0 + 32 * i < nv) {
          const size_t at = dst + static_cast<size_t>(v0 + 32 * i) * VEC;
          float o[VEC];
          Piece<VEC, false> before;
          if (a.add) before.load(a.add, at);
#pragma unroll
          for (int e = 0; e < VEC; ++e) o[e] = a.add ? fmaf(a.scale, acc[i][e], before[e]) : a.scale * acc[i][e];
          store_vec<VEC, true>(a.d_table, at, o);
        }
    }
    start += n;
  }
}

size_t padded(size_t n) { return (n + 255) / 256 * 256; }

template <int VEC, bool kF32>
cudaError_t launch_sums(const SumArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.chunks > 0) {
    e = launch_kernel(embedding_chunk_kernel<VEC, kF32>, dim3((a.chunks + 7) / 8), dim3(256), 0, s, true, a);
    if (e != cudaSuccess) return e;
  }
  const int warps = (a.V + kRowsPerWarp - 1) / kRowsPerWarp;
  return launch_kernel(embedding_rows_kernel<VEC, kF32>, dim3((warps + 7) / 8), dim3(256), 0, s, a.T > 0, a);
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingArgs& a, cudaStream_t s) {
  return a.D % 8 == 0 ? launch_fwd<8>(a, s) : launch_fwd<1>(a, s);
}

size_t embedding_bwd_scratch_bytes(int T, int V, int D) {
  const SortPlan p = sort_plan(T, V);
  return padded(static_cast<size_t>(p.passes) * p.blocks * (sizeof(uint32_t) << p.bits)) +
         4 * padded(static_cast<size_t>(T) * sizeof(uint32_t)) + padded(static_cast<size_t>(p.chunks) * D * sizeof(float));
}

cudaError_t launch_embedding_bwd(const EmbeddingBwdArgs& a, void* scratch, cudaStream_t s) {
  const SortPlan p = sort_plan(a.T, a.V);
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
  q.passes = p.passes;
  q.hist = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(p.passes) * p.blocks * (sizeof(uint32_t) << p.bits)));
  uint32_t* lists[4];
  for (auto& l : lists) l = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(a.T) * sizeof(uint32_t)));
  float* part = reinterpret_cast<float*>(take(static_cast<size_t>(p.chunks) * a.D * sizeof(float)));
  cudaError_t e = cudaSuccess;
  if (a.T > 0) {
    e = launch_kernel(embedding_hist_kernel, dim3(p.blocks), dim3(kSortThreads), 0, s, false, q);
    for (int i = 0; i < p.passes && e == cudaSuccess; ++i) {
      q.pass = i;
      q.key_out = lists[2 * (i & 1)];
      q.tok_out = lists[2 * (i & 1) + 1];
      e = launch_kernel(embedding_sort_kernel, dim3(p.blocks), dim3(kSortThreads), 0, s, true, q);
      q.key_in = q.key_out;
      q.tok_in = q.tok_out;
    }
    if (e != cudaSuccess) return e;
  }
  const SumArgs m{a.d_out, a.add, q.key_in, q.tok_in, part, a.d_table, a.scale, a.T, a.V, a.D, p.chunk, p.chunks};
  if (a.D % 8 == 0) return a.d_fp32 ? launch_sums<8, true>(m, s) : launch_sums<8, false>(m, s);
  return a.d_fp32 ? launch_sums<1, true>(m, s) : launch_sums<1, false>(m, s);
}

}  // namespace moe
