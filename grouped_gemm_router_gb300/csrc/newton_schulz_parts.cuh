// How newton_schulz_small.cu cuts a matrix into the parts of a cluster's CTAs,
// and the order in which a CTA's threads go through their part in memory.
// Index arithmetic only, for the host as well.
#pragma once

#include "moe_device.cuh"

namespace moe {

namespace {

constexpr int kRowsMax = 128;                    // most rows (short side)
constexpr int kSlice = 256;                      // most columns of a CTA
constexpr int kMaxCluster = 8;
constexpr int kThreads = 512;                    // 16 warps: 4 lane quarters x 4 column quarters
constexpr int kPitch = kSlice + 4;               // stash: 16-byte pieces of 8 rows meet no bank conflict

// CTAs of a matrix with n columns, the columns of each, and those that CTA
// `rank` has inside the matrix.  The first is a power of two and the second a
// multiple of 64, so the last CTAs may have none (n = 1025: 8 of 192).
__host__ MOE_DEV int cluster_ranks(int n) {
  int ranks = 1;
  while (ranks * kSlice < n) ranks *= 2;
  return ranks;
}
__host__ MOE_DEV int slice_columns(int n, int ranks) { return ((n + ranks - 1) / ranks + 63) / 64 * 64; }
__host__ MOE_DEV int slice_width(int n, int slice, int rank) {
  const int left = n - rank * slice;
  return left < 0 ? 0 : left < slice ? left : slice;
}

// The CTA's part of a matrix in memory order, runs of VEC elements, batch(VEC)
// a thread at a time.  Four-element runs are for matrices that lie in memory as
// X does; in a tall one a run would be a column of the stash, and single
// elements meet fewer bank conflicts (4 lanes a bank).  In the stash the run
// at memory row r, place x starts at element r * sr + x * sx.  A part without
// columns has no rows either, so that no run of it is visited.
__host__ __device__ constexpr int batch(int vec) { return vec == 4 ? 4 : 16; }
struct Part {
  int rows, len, shift;  // memory rows, elements of one, 2^shift runs cover it
  int sr, sx;
  int first, pitch;      // element of the matrix where the part starts, and between rows
};
template <int VEC>
__host__ MOE_DEV Part part_of(bool tall, int m, int n, int c0, int width) {
  Part q;
  q.rows = tall ? width : width > 0 ? m : 0;
  q.len = tall ? m : width;
  q.shift = 0;
  while ((VEC << q.shift) < q.len) ++q.shift;
  q.sr = tall ? 1 : kPitch;
  q.sx = tall ? kPitch : 1;
  q.first = tall ? c0 * m : c0;
  q.pitch = tall ? m : n;
  return q;
}
__host__ MOE_DEV int run_count(const Part& q) { return q.rows << q.shift; }

// Where run s starts: element `at` of the matrix, element `spot` of the stash.
// A run past the end of a row or of the part repeats the part's first one,
// with spot = -1: it is loaded and not used.
template <int VEC>
__host__ MOE_DEV void place_run(const Part& q, int s, int& at, int& spot) {
  const int r = s >> q.shift, x = (s & ((1 << q.shift) - 1)) * VEC;
  const bool in = r < q.rows && x < q.len;
  at = in ? q.first + r * q.pitch + x : q.first;
  spot = in ? r * q.sr + x * q.sx : -1;
}

}  // namespace

}  // namespace moe
