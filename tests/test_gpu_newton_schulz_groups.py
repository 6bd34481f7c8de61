"""Newton-Schulz of more matrices than are worked on at a time, each with values
of its own: every CTA counts many tiles and reuses their places, and a matrix
must not see another's parts across the groups.  The tile width alone decides
the order of a matrix's sums, so a matrix has the bits that it has in a smaller
call with tiles of the same width, and the same bits every time."""
import numpy as np
import pytest
import torch

from _train_ref import newton_schulz

pytestmark = pytest.mark.gpu

C = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def _stack(B, rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    # each matrix has a strength and a direction of its own
    x = torch.randn(B, rows, cols, generator=g, device="cuda")
    return 1e-3 * torch.exp(torch.randn(B, 1, 1, generator=g, device="cuda")) * x


# (matrices, rows, cols, matrices of the smaller calls): 77 go in groups of 26,
# 26 and 25, 999 in six of 167 and less; the smaller calls are the fewest that
# still take tiles of 256 columns (more than two waves of narrow ones)
@pytest.mark.parametrize("B,rows,cols,some", [(77, 768, 1536, 9), (999, 129, 200, 160), (40, 1536, 768, 9)])
def test_groups_of_different_matrices(moe, B, rows, cols, some):
    g = _stack(B, rows, cols, B)
    o = moe.newton_schulz(g)
    torch.cuda.synchronize()
    assert moe.device_error() == 0
    for first in [*range(0, B - some, some), B - some]:
        part = moe.newton_schulz(g[first:first + some].clone())
        assert torch.equal(part, o[first:first + some]), first
    for e in (0, 25, 26, B - 1):       # on both sides of a border, against the definition
        ref = newton_schulz(f64(g[e]), [C] * 5, 1e-7)
        # 4e-3 in the 2-norm: fp16 operands (1.6e-3) and the bf16 result, see test_gpu_newton_schulz.py
        assert np.sqrt(((f64(o[e]) - ref) ** 2).sum() / (ref ** 2).sum()) <= 4e-3
    for _ in range(10):
        assert torch.equal(o, moe.newton_schulz(g))


def test_parts_counted_by_the_warps_themselves(moe):
    """So few tiles that each epilogue warp counts its own part."""
    for B, rows, cols in ((1, 600, 900), (3, 200, 333), (2, 1001, 363)):
        g = _stack(B, rows, cols, rows)
        o = moe.newton_schulz(g)
        for _ in range(30):
            assert torch.equal(o, moe.newton_schulz(g))
        for e in range(B):
            assert torch.equal(o[e], moe.newton_schulz(g[e].clone()))
    torch.cuda.synchronize()
    assert moe.device_error() == 0
