"""Embedding lookup and its gradient on the GPU against 64-bit statements.

Tolerances: the lookup is one product in fp32 and one rounding, so a value is
off by 2^-24 of itself, and 2^-8 where it is stored as bf16.  A gradient is a
sum of n terms in fp32, n - 1 roundings of partial sums that are at most the
sum of the magnitudes, and up to two more: (n + 2) 2^-24 of that sum."""
import numpy as np
import pytest
import torch

import _lm_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


def _np(t):
    return t.detach().cpu().double().numpy() if t.dtype != BF else t.detach().float().cpu().double().numpy()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("table_type,out_type,index", [(BF, None, torch.int64), (BF, F32, torch.int32), (F32, BF, torch.int64),
                                                       (F32, None, torch.int32)])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 7, 8192), (3, 5, 64), (16, 1000, 768), (33, 10, 1005), (1001, 5003, 72),
                                   (5000, 300, 768), (0, 4, 64), (4097, 9, 8)])
def test_forward(moe, T, V, D, table_type, out_type, index):
    g = _gen(T + V + D)
    table = torch.randn(V, D, generator=g, device="cuda").to(table_type)
    ids = torch.randint(-2, V + 2, (T,), generator=g, device="cuda", dtype=index)
    out = moe.embedding_forward(ids, table, scale=1.7, out_type=out_type)
    assert out.dtype == (out_type or table_type) and out.shape == (T, D)
    want = ref.embedding(ids.cpu().numpy(), _np(table), np.float64(np.float32(1.7)))
    eps = 2.0 ** -24 + (2.0 ** -8 if out.dtype == BF else 0)
    assert (np.abs(_np(out) - want) <= eps * np.abs(want) * 1.0001).all()


def _check_backward(moe, ids, d_out, V, scale, add):
    got = moe.embedding_backward(d_out, ids, V, scale=scale, add=add)
    assert got.dtype == F32 and got.shape == (V, d_out.shape[1])
    i, d, a = ids.cpu().numpy(), _np(d_out), None if add is None else _np(add)
    s = float(np.float32(scale))
    want = ref.embedding_grad(d, i, V, s, a)
    size = ref.embedding_grad(np.abs(d), i, V, abs(s), None if a is None else np.abs(a))
    n = np.bincount(i[(i >= 0) & (i < V)].astype(np.int64), minlength=V)[:, None] + 2
    assert (np.abs(_np(got) - want) <= n * 2.0 ** -24 * size).all()
    assert torch.equal(moe.embedding_backward(d_out, ids, V, scale=scale, add=add), got)  # the same bits every time
    return got


@pytest.mark.parametrize("grad_type,with_add,index", [(BF, False, torch.int64), (BF, True, torch.int32),
                                                      (F32, False, torch.int32), (F32, True, torch.int64)])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 300, 64), (31, 3, 8), (32, 1, 768), (33, 1, 1005), (64, 2, 72), (0, 5, 64),
                                   (0, 3, 13), (700, 2000, 768), (1001, 5003, 1005), (2049, 70, 8192), (5000, 1 << 20, 8),
                                   (9000, 40, 264), (2048, 50, 40), (32768, 300, 24), (32769, 70000, 13), (50000, 262144, 16)])
def test_backward(moe, T, V, D, grad_type, with_add, index):
    g = _gen(T + V + D)
    ids = torch.randint(-1, V + 1, (T,), generator=g, device="cuda", dtype=index)
    d_out = torch.randn(T, D, generator=g, device="cuda").to(grad_type)
    add = torch.randn(V, D, generator=g, device="cuda").bfloat16() if with_add else None
    _check_backward(moe, ids, d_out, V, -1.3, add)


@pytest.mark.parametrize("D", [24, 40, 13])
def test_runs_of_every_length(moe, D):
    """Tokens that come 0 to 100 times, so that runs begin and end everywhere in
    the chunks of 32, and some that come thousands of times; most of them last."""
    counts = list(range(101)) + [0, 0, 3000, 1, 31, 1024, 0, 33, 2048, 95]
    ids = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))].to("cuda")
    d_out = torch.randn(len(ids), D, generator=_gen(2), device="cuda")
    _check_backward(moe, ids, d_out, len(counts) + 3, 0.5, None)
    _check_backward(moe, torch.full_like(ids, -1), d_out, 7, 0.5, None)   # no token at all
    _check_backward(moe, torch.full_like(ids, 6), d_out, 7, 0.5, None)    # one token only


def test_many_tokens_and_blocks(moe):
    """More tokens than 128 sort blocks of 2048, three passes of the sort, long
    chunks; sums of whole numbers are exact in any order."""
    T, V, D = 300001, (1 << 20) + 5, 16
    g = _gen(3)
    ids = torch.where(torch.rand(T, generator=g, device="cuda") < 0.3, 5,
                      torch.randint(0, V, (T,), generator=g, device="cuda"))
    d_out = torch.randint(-8, 9, (T, D), generator=g, device="cuda").float()
    want = torch.zeros(V, D, device="cuda").index_add_(0, ids, d_out)
    assert torch.equal(moe.embedding_backward(d_out, ids, V), want)


@pytest.mark.parametrize("T,V", [(512, 3), (513, 3000), (4096, 100), (4097, 600000), (40000, 700), (65536, 900), (65537, 900)])
def test_long_runs_of_odd_rows(moe, T, V):
    """Lists at the edges of the on-chip sorts and past them, rows without
    16-byte pieces, ids that come thousands of times."""
    g = _gen(T)
    D = 21
    ids = (torch.rand(T, generator=g, device="cuda") ** 4 * V).long()
    _check_backward(moe, ids, torch.randn(T, D, generator=g, device="cuda"), V, 2.0,
                    torch.randn(V, D, generator=g, device="cuda").bfloat16())


@pytest.mark.parametrize("T,V,D", [(1, 2, 4097), (40, 2, 8192), (562, 3, 3346), (2048, 9, 2056), (2049, 1, 8191), (3000, 5, 2056)])
@pytest.mark.parametrize("grad_type,with_add", [(BF, True), (F32, False)])
def test_few_tokens_of_wide_rows(moe, T, V, D, grad_type, with_add):
    """A row's columns are shared among blocks, those of long runs too."""
    g = _gen(T)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    add = torch.randn(V, D, generator=g, device="cuda").bfloat16() if with_add else None
    _check_backward(moe, ids, torch.randn(T, D, generator=g, device="cuda").to(grad_type), V, 0.7, add)


def test_calls_from_several_host_threads(moe):
    from concurrent.futures import ThreadPoolExecutor
    g = _gen(10)
    ids = torch.randint(0, 500, (3000,), generator=g, device="cuda")
    d_out = torch.randn(3000, 64, generator=g, device="cuda").bfloat16()
    want = moe.embedding_backward(d_out, ids, 500)
    torch.cuda.synchronize()

    def work(_):
        with torch.cuda.stream(torch.cuda.Stream()):
            out = [moe.embedding_backward(d_out, ids, 500) for _ in range(10)]
            torch.cuda.current_stream().synchronize()
        return all(torch.equal(o, want) for o in out)

    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(work, range(8)))


def test_offsets_past_32_bits(moe):
    """A table of more than 2^31 elements: its last rows."""
    V, D = (1 << 18) + 3, 8192
    table = torch.zeros(V, D, dtype=BF, device="cuda")
    table[-2:] = torch.arange(2 * D, device="cuda").view(2, D).remainder(251).bfloat16()
    ids = torch.tensor([V - 1, V - 2, 0, V], device="cuda")
    out = moe.embedding_forward(ids, table)
    assert torch.equal(out[:2], table[-2:].flip(0)) and not out[2:].any()
    del table
    d = torch.ones(4, D, dtype=BF, device="cuda")
    g = moe.embedding_backward(d, ids, V)
    assert (g[-2:] == 1).all() and (g[0] == 1).all() and not g[1:-2].any()


def test_infinities_stay_in_their_rows(moe):
    ids = torch.tensor([1, 2, -1, 1], device="cuda")
    d = torch.ones(4, 40, device="cuda")
    d[1], d[2] = float("inf"), float("nan")
    g = moe.embedding_backward(d, ids, 4)
    assert (g[1] == 2).all() and torch.isinf(g[2]).all() and not g[0].any() and not g[3].any()


@pytest.mark.parametrize("D", [40, 13])
def test_views_that_start_anywhere(moe, D):
    g = _gen(5)

    def view(t):
        buf = torch.full((t.numel() + 2,), 7, dtype=t.dtype, device="cuda")
        v = buf[1:-1].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 16
        return v

    ids = torch.randint(0, 50, (60,), generator=g, device="cuda")
    table = torch.randn(50, D, generator=g, device="cuda").bfloat16()
    d_out, add = torch.randn(60, D, generator=g, device="cuda").bfloat16(), torch.randn(50, D, generator=g, device="cuda").bfloat16()
    f, b = moe.embedding_forward(ids, table), moe.embedding_backward(d_out, ids, 50, add=add)
    assert torch.equal(moe.embedding_forward(view(ids), view(table)), f)
    assert torch.equal(moe.embedding_backward(view(d_out), view(ids), 50, add=view(add)), b)


def test_captured_and_on_streams(moe):
    """A captured step replays on new contents; two streams with workspaces of
    their own do not meet."""
    g = _gen(6)
    T, V, D = 3000, 900, 128
    sets = [(torch.randint(0, V, (T,), generator=g, device="cuda"), torch.randn(T, D, generator=g, device="cuda").bfloat16())
            for _ in range(3)]
    want = [moe.embedding_backward(d, i, V) for i, d in sets]
    ids, d_out = (t.clone() for t in sets[0])
    ws = torch.empty(moe.embedding_backward_workspace_size(T, V, D), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        moe.embedding_backward(d_out, ids, V, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = moe.embedding_backward(d_out, ids, V, workspace=ws)
        for (i, d), w in zip(sets, want):
            ids.copy_(i)
            d_out.copy_(d)
            graph.replay()
            s.synchronize()
            assert torch.equal(got, w)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    out = []
    for st, (i, d) in zip(streams, sets):
        with torch.cuda.stream(st):
            out.append([moe.embedding_backward(d, i, V) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for os, w in zip(out, want) for o in os)


@pytest.mark.parametrize("T,D", [(5000, 768), (70000, 40)])
def test_long_runs_in_a_captured_graph(moe, T, D):
    """Replays find other long runs, many, few or none, in whatever order, and
    give the bits of a call of its own."""
    g = _gen(12)
    V = 4000
    skew = [(torch.rand(T, generator=g, device="cuda") ** p * V).long() for p in (6, 1.5)]
    sets = [skew[0], torch.arange(T, device="cuda") % V, torch.full((T,), 7, device="cuda"), skew[1],
            torch.full((T,), -1, device="cuda"), skew[0].flip(0).contiguous()]
    d_out = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    want = [moe.embedding_backward(d_out, i, V) for i in sets]
    for i, w in zip(sets, want):
        assert all(torch.equal(moe.embedding_backward(d_out, i, V), w) for _ in range(3))
    ids = sets[0].clone()
    ws = torch.full((moe.embedding_backward_workspace_size(T, V, D),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        moe.embedding_backward(d_out, ids, V, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = moe.embedding_backward(d_out, ids, V, workspace=ws)
        for i, w in list(zip(sets, want)) * 2:
            ids.copy_(i)
            graph.replay()
            s.synchronize()
            assert torch.equal(got, w)
