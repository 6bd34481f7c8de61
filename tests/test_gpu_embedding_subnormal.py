"""Embedding gradients next to 2^-126: sums, and what is added to them, keep
their subnormal values whichever way a row takes (a window, a long run listed or
not, 16-byte pieces or single elements)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [40, 13])
@pytest.mark.parametrize("T", [8, 300, 5000])
@pytest.mark.parametrize("with_add", [False, True])
def test_subnormal_sums(moe, T, D, grad, with_add):
    """Whole multiples of 2^-133 below 2^-126 in all: every sum is exact."""
    g = torch.Generator(device="cuda").manual_seed(T + D)
    V, unit = 9, 2.0 ** -133
    ids = torch.arange(T, device="cuda") % 5
    if T > 8:
        ids[20:] = 7  # a long run
    few = (torch.rand(T, generator=g, device="cuda") < 30 / T).double()[:, None]  # most rows are zero: sums stay small
    d = torch.randint(-3, 4, (T, D), generator=g, device="cuda").double() * few
    a = torch.randint(-60, 61, (V, D), generator=g, device="cuda").double()
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids, d) + (a if with_add else 0)
    assert want.abs().max() < 2 ** 8 and want.any()
    d_out, add = (d * unit).to(grad), (a * unit).bfloat16()
    assert torch.equal(d_out.double(), d * unit) and torch.equal(add.double(), a * unit)
    got = moe.embedding_backward(d_out, ids, V, add=add if with_add else None)
    assert torch.equal(got.double(), want * unit)
