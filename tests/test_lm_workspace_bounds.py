"""Workspaces of the vocabulary losses against the bound that the header states:
forward a pair of floats for each half of each run of 256 columns or more, and
the teacher's keys; backward dz (2 T V bytes, at most the larger of 4 GiB and 4096 T)
and fp32 parts of dx and dW where their reductions are cut."""
import pytest


@pytest.fixture(scope="module")
def N():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import _native
    return _native


GIB = 1 << 30


@pytest.mark.parametrize("T", [1, 127, 4096, 1 << 18, 1 << 20, (1 << 20) + 1, 1 << 22, (1 << 24) - 5, 1 << 24])
@pytest.mark.parametrize("V", [1, 300, 5003, 50001, 131072, 1 << 22])
def test_backward_size(N, T, V):
    D = 64
    n = N.lib.moe_vocab_backward_workspace_size(T, D, V, 0)
    dz = min(2 * T * (-(-V // 64) * 64), max(4 * GIB, 4096 * T))
    parts = 76 * 4 * D * (T + V)  # each reduction is cut for at most as many pairs as there are
    assert 0 < n <= dz + parts + 4096
    # as few pieces as there can be, all alike: of up to 2048 columns, V / ceil(V / 2048) >= 1024 of them where V > 2048
    assert n >= min(2 * T * V, 2 * T * 1024)
    if T <= 1 << 20:
        assert n <= 4 * GIB + parts + 4096


def test_largest_size(N):
    """2^24 tokens: 2048 columns of dz are 64 GiB, and the dx that the pieces add up is T D floats."""
    T, D, V = 1 << 24, 64, 1 << 17
    n = N.lib.moe_vocab_backward_workspace_size(T, D, V, 0)
    assert 64 * GIB + 4 * T * D <= n <= 64 * GIB + 4 * T * D * 2


@pytest.mark.parametrize("T,V", [(1, 1 << 22), (4096, 50001), (1 << 24, 131072)])
def test_forward_size(N, T, V):
    """(maximum, sum) of two halves of each run of at least 256 columns."""
    rows = -(-T // 32) * 32
    for K in (0, 7):
        n = N.lib.moe_vocab_forward_workspace_size(T, 64, V, K)
        assert 0 < n <= 16 * rows * -(-V // 256) + 4 * T * max(K, 1) + 1024
