"""Where the on-chip Newton-Schulz kernel reads and writes a matrix: the index
arithmetic of csrc/newton_schulz_parts.cuh, run on the host for every CTA and
thread.  Every element that a thread touches has to lie inside the matrix, one
row or many, and every element has to be visited exactly once."""
import subprocess

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "newton_schulz_parts.cuh"
using namespace moe;

static long bad = 0;

template <int VEC>
void walk(bool tall, int m, int n) {
  const int ranks = cluster_ranks(n), slice = slice_columns(n, ranks);
  const long size = static_cast<long>(m) * n;
  std::vector<int> seen(size, 0);
  for (int rank = 0; rank < ranks; ++rank) {
    const Part q = part_of<VEC>(tall, m, n, rank * slice, slice_width(n, slice, rank));
    const int total = run_count(q);
    for (int t = 0; t < kThreads; ++t)
      for (int s0 = t; s0 < total; s0 += kThreads * batch(VEC))
        for (int k = 0; k < batch(VEC); ++k) {
          int at, spot;
          place_run<VEC>(q, s0 + k * kThreads, at, spot);
          if (at < 0 || at + VEC > size || spot >= kRowsMax * kPitch) {
            if (++bad <= 5) std::printf("%d x %d tall %d VEC %d rank %d reads %d of %ld\n", m, n, tall, VEC, rank, at, size);
            continue;
          }
          if (spot >= 0)
            for (int j = 0; j < VEC; ++j) ++seen[at + j];
        }
  }
  for (long i = 0; i < size; ++i)
    if (seen[i] != 1 && ++bad <= 5) std::printf("%d x %d tall %d VEC %d element %ld visited %d times\n", m, n, tall, VEC, i, seen[i]);
}

int main() {
  const int rows[] = {1, 2, 3, 4, 17, 64, 65, 127, 128};
  for (int m : rows)
    for (int n = m; n <= kSlice * kMaxCluster; n += m <= 4 ? 1 : 37) {
      walk<1>(false, m, n);
      walk<1>(true, m, n);
      if (m % 4 == 0 && n % 4 == 0) walk<4>(false, m, n);
    }
  std::printf("%ld accesses out of place\n", bad);
  return bad != 0;
}
"""


def test_every_access_lies_in_the_matrix(tmp_path):
    from grouped_gemm_router_gb300 import build
    src, exe = tmp_path / "parts.cu", tmp_path / "parts"
    src.write_text(PROGRAM)
    r = subprocess.run([build._nvcc(), *build.ARCH, "-O2", "-std=c++17", f"-I{build.CSRC}", str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
