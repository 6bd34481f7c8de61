"""How the vocabulary products are cut and dealt (csrc/vocab_plan.cuh), run on
the host for every CTA pair: each tile, and each k block of each tile, belongs
to exactly one unit of one pair, no unit is empty, the runs of the forward
write pairs that lie in the workspace, and the pieces cover the vocabulary."""
import subprocess

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "vocab_plan.cuh"
using namespace moe;

static long bad = 0;
#define CHECK(ok, ...) do { if (!(ok) && ++bad <= 10) { std::printf(__VA_ARGS__); std::printf("\n"); } } while (0)

template <int kMode>
void tiles(const VocabWork& w, int npairs, int runs, const char* what) {
  std::vector<int> seen(static_cast<size_t>(w.nmt) * w.nnt, 0);
  npairs = std::min(npairs, w.items);
  for (int pair = 0; pair < npairs; ++pair) {
    Walk<kMode> walk;
    Unit u;
    int m = -1, slot = -1, open = 0, next = 0;
    while (walk.next(w, pair, npairs, u)) {
      CHECK(u.m >= 0 && u.m < w.nmt && u.n >= 0 && u.n < w.nnt, "%s: tile %d %d", what, u.m, u.n);
      ++seen[static_cast<size_t>(u.m) * w.nnt + u.n];
      CHECK(u.kb0 == 0 && u.kb1 == w.nkb[0] && u.kb1 > 0, "%s: k blocks", what);
      CHECK(u.slot >= 0 && u.slot < runs, "%s: slot %d of %d", what, u.slot, runs);
      if (u.first) { CHECK(!open, "%s: a run begins inside another", what); m = u.m; slot = u.slot; open = 1; next = u.n; }
      CHECK(open && u.m == m && u.slot == slot && u.n == next, "%s: a run is broken", what);
      ++next;
      if (u.last) open = 0;
    }
    CHECK(!open, "%s: a run has no end", what);
  }
  for (int s : seen) CHECK(s == 1, "%s: a tile is computed %d times", what, s);
}

void units(const VocabWork& w, int npairs, const char* what) {
  std::vector<int> seen[2];
  for (int i = 0; i < 2; ++i) seen[i].assign(static_cast<size_t>(w.tiles_m[i]) * w.tiles_n * w.nkb[i], 0);
  npairs = std::min(npairs, w.n_units[0] + w.n_units[1]);
  for (int pair = 0; pair < npairs; ++pair) {
    Walk<kGrad> walk;
    Unit u;
    while (walk.next(w, pair, npairs, u)) {
      const int i = u.which;
      CHECK(u.m >= 0 && u.m < w.tiles_m[i] && u.n >= 0 && u.n < w.tiles_n && u.split >= 0 && u.split < w.splits[i],
            "%s: unit", what);
      CHECK(u.kb0 >= 0 && u.kb0 < u.kb1 && u.kb1 <= w.nkb[i], "%s: k blocks %d to %d", what, u.kb0, u.kb1);
      for (int k = u.kb0; k < u.kb1; ++k) ++seen[i][(static_cast<size_t>(u.m) * w.tiles_n + u.n) * w.nkb[i] + k];
    }
  }
  for (int i = 0; i < 2; ++i)
    for (int s : seen[i]) CHECK(s == 1, "%s: a block of %s is added %d times", what, i ? "dW" : "dx", s);
}

int main() {
  const int ts[] = {1, 2, 255, 256, 257, 1001, 4096, 20001, 32768, 300000};
  const int ds[] = {64, 192, 768, 2048, 8192};
  const int vs[] = {1, 63, 100, 256, 257, 5003, 50001, 131072, 262145};
  for (int T : ts) for (int V : vs) for (int npairs : {1, 3, 74, 76}) {
    const ForwardPlan f = forward_plan(T, V);
    char what[80];
    std::snprintf(what, sizeof what, "T %d V %d pairs %d", T, V, npairs);
    if (static_cast<long>(f.nmt) * f.nnt > 200000) continue;
    CHECK(f.rows_padded >= T && f.run * f.runs >= f.nnt, "%s: plan", what);
    tiles<kStats>(forward_work(f, 768), npairs, f.runs, what);
    for (int D : ds) {
      const BackwardPlan b = backward_plan(T, D, V);
      CHECK(b.piece > 0 && static_cast<long>(b.piece) * b.pieces >= V && static_cast<long>(b.piece) * (b.pieces - 1) < V, "%s: pieces", what);
      CHECK(b.pieces == 1 || b.piece % kTile == 0, "%s: piece %d", what, b.piece);
      CHECK(b.piece % 64 == 0 && b.splits_x >= 1 && b.splits_w >= 1, "%s: plan", what);
      CHECK(b.piece <= 8 * kTile || static_cast<size_t>(b.piece) * T * 2 <= kPieceBytes + static_cast<size_t>(T) * 2 * kTile, "%s: piece of %d", what, b.piece);
      for (int i = 0; i < b.pieces; i += std::max(1, b.pieces - 1)) {
        const int Vc = std::min(b.piece, V - i * b.piece);
        const VocabWork d = dz_work(b, D, Vc);
        tiles<kDz>(d, npairs, ceil_div(d.nnt, d.run), what);
        const VocabWork w = grad_work(b, T, Vc);
        CHECK(w.splits[0] <= b.splits_x && w.splits[1] <= b.splits_w, "%s: splits", what);
        CHECK(i > 0 || w.splits[0] == b.splits_x, "%s: the first piece writes every part", what);
        units(w, npairs, what);
      }
    }
  }
  std::printf("%ld bad\n", bad);
  return bad != 0;
}
"""


def test_every_block_is_computed_once(tmp_path):
    from grouped_gemm_router_gb300 import build as b
    src = tmp_path / "plan.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "plan"
    subprocess.run([b._nvcc(), "-std=c++17", "-O2", f"-I{b.CSRC}", f"-I{b.INCLUDE}", *b.ARCH, str(src), "-o", str(exe)],
                   check=True, capture_output=True, text=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout
