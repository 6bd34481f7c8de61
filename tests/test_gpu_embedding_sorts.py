"""Lists of 4097 to 65536 tokens, which a cluster of 16 blocks sorts on chip, as
on a device that holds no such cluster: the same bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


@pytest.mark.parametrize("T,V,D", [(1, 3, 8), (512, 40, 8), (4096, 700, 16), (4097, 3, 24), (5000, 1 << 20, 8), (8193, 700, 13),
                                   (32768, 50001, 24), (40001, 1 << 22, 1), (65535, 9, 40), (65536, 70000, 16)])
@pytest.mark.parametrize("with_add", [False, True])
def test_without_large_clusters(moe, T, V, D, with_add):
    from grouped_gemm_router_gb300 import _native as N
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = (torch.rand(T, generator=g, device="cuda") ** 3 * (V + 2)).long() - 1
    d_out = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    add = torch.randn(V, D, generator=g, device="cuda").bfloat16() if with_add else None
    want = moe.embedding_backward(d_out, ids, V, scale=0.5, add=add)
    n = moe.embedding_backward_workspace_size(T, V, D)
    ws = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((V + 1, D), 7.0, device="cuda")
    before = N.lib.moe_launch_count()
    st = N.lib.moe_selftest_embedding_by_passes(d_out.data_ptr(), N.MOE_BF16, ids.data_ptr(), N.MOE_I64, 0.5,
                                                None if add is None else add.data_ptr(), T, V, D, out.data_ptr(),
                                                ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert st == N.MOE_OK
    if T > 4096:  # histogram, a launch a pass, fill, rows, long runs
        assert N.lib.moe_launch_count() - before == 4 + (3 if V >= 1 << 18 else 2 if V >= 1 << 9 else 1)
    assert torch.equal(out[:V], want) and (out[V] == 7).all() and (ws[n:] == 77).all()
    # and in 64 bits: sums of bf16 rows, at most T terms rounded by 2^-24
    known = (ids >= 0) & (ids < V)
    exact = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(exact)
    if with_add:
        exact += add.double()
        size += add.double().abs()
    exact.index_add_(0, ids[known], 0.5 * d_out[known].double())
    size.index_add_(0, ids[known], 0.5 * d_out[known].double().abs())
    count = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, ids[known], torch.ones_like(ids[known]).double())
    assert ((want.double() - exact).abs() <= (count + 2)[:, None] * 2.0 ** -24 * size).all()


def test_small_scratch_is_refused(moe):
    """The size covers both ways to sort, and one byte less is refused."""
    from grouped_gemm_router_gb300 import _native as N
    T, V, D = 5000, 700, 8
    n = moe.embedding_backward_workspace_size(T, V, D)
    fake = 0x100000
    for call in (N.lib.moe_embedding_backward, N.lib.moe_selftest_embedding_by_passes):
        assert call(fake, 0, fake, 1, 1.0, None, T, V, D, fake, fake, n - 1, None) == N.MOE_ERR_WORKSPACE
